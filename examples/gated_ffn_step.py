"""A feed-forward block with a gated linear unit, trained and served.

    python examples/gated_ffn_step.py            # needs an MI355X and the built library

    Y = act(X W_gate) * (X W_up)                 tp_gated_linear
    out = Y W_down + bias + X                    tp_linear (bias and residual in the product)

Training: forward, a squared-error loss against a teacher block, both backward passes, the global gradient norm
with clipping, and a plain gradient step on fp32 main weights; the loss has to fall.  Serving: the trained block
run for one token at a time through prepared calls, which has to give the batch's rows.
"""
from __future__ import annotations

import math
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import sharded_gemm_amd as tp  # noqa: E402

BF16 = torch.bfloat16


class GatedFFN:
    """The block's weights (fp32 main copies, bf16 working copies), gradients and workspaces for one batch size."""

    def __init__(self, tokens, width, inner, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def weight(*shape):
            return torch.randn(shape, generator=g, device="cuda") / math.sqrt(shape[0])
        self.main = dict(gate=weight(width, inner), up=weight(width, inner), down=weight(inner, width),
                         bias=torch.zeros(width, device="cuda"))
        self.grads = {k: torch.zeros_like(v) for k, v in self.main.items()}
        self.refresh()

        def rows(cols, dtype=BF16):
            return torch.empty((tokens, cols), dtype=dtype, device="cuda")
        self.gate, self.up, self.y, self.out = rows(inner), rows(inner), rows(inner), rows(width)
        self.d_y, self.d_x = rows(inner), rows(width, torch.float32)
        self.ws_down = tp.tp_linear_backward_ws(self.y, self.w["down"], self.out, dbias=self.grads["bias"])
        self.ws_gated = tp.tp_gated_linear_backward_ws(self.out, self.y)
        self.parts, self.norm = tp.tp_grad_parts(), torch.empty(1, device="cuda")

    def refresh(self):
        self.w = {k: v.to(BF16) for k, v in self.main.items() if k != "bias"}

    def forward(self, x):
        tp.tp_gated_linear(x, self.w["gate"], self.w["up"], self.y, gate_out=self.gate, up_out=self.up)
        tp.tp_linear(self.y, self.w["down"], self.out, bias=self.main["bias"], residual=x)
        return self.out

    def backward(self, x, d_out):
        """Fills self.grads (fp32) and self.d_x, the gradient at the block's input without its residual branch."""
        tp.tp_linear_backward(self.y, self.w["down"], d_out, dX=self.d_y, dW=self.grads["down"],
                              dbias=self.grads["bias"], ws=self.ws_down)
        tp.tp_gated_linear_backward(x, self.w["gate"], self.w["up"], self.gate, self.up, self.d_y, dX=self.d_x,
                                    dW_gate=self.grads["gate"], dW_up=self.grads["up"], ws=self.ws_gated)

    def clip(self, max_norm):
        grads = list(self.grads.values())
        tp.tp_grad_sumsq(grads, self.parts)
        tp.tp_grad_clip(grads, None, self.parts, max_norm=max_norm, norm_out=self.norm)
        return self.norm

    def step(self, rate):
        for k, v in self.main.items():
            v.sub_(self.grads[k], alpha=rate)
        self.refresh()


def train(tokens=512, width=256, inner=384, steps=30, rate=30.0, max_norm=0.05, seed=0):
    """Losses of the steps, the norms, and the trained block with its input."""
    g = torch.Generator(device="cuda").manual_seed(seed + 100)
    x = torch.randn((tokens, width), generator=g, device="cuda").to(BF16)
    target = GatedFFN(tokens, width, inner, seed + 1).forward(x).float()
    block = GatedFFN(tokens, width, inner, seed + 2)
    losses, norms = [], []
    for _ in range(steps):
        diff = block.forward(x).float() - target
        losses.append(diff.square().mean())
        block.backward(x, (diff * (2.0 / diff.numel())).to(BF16))
        norms.append(block.clip(max_norm).clone())
        block.step(rate)
    return [float(v) for v in losses], [float(v) for v in norms], block, x


def serve(block, x):
    """The block's output one token at a time, through prepared calls."""
    tok = torch.empty((1, x.shape[1]), dtype=BF16, device="cuda")
    y = torch.empty((1, block.y.shape[1]), dtype=BF16, device="cuda")
    out = torch.empty_like(tok)
    up = tp.tp_gated_linear(tok, block.w["gate"], block.w["up"], y, prepare=True)
    down = tp.tp_linear(y, block.w["down"], out, bias=block.main["bias"], residual=tok, prepare=True)
    rows = []
    for t in range(x.shape[0]):
        tok.copy_(x[t:t + 1])
        up()
        down()
        rows.append(out.clone())
    return torch.cat(rows)


def main():
    losses, norms, block, x = train()
    print("loss %.4f -> %.4f, gradient norm %.4f -> %.4f" % (losses[0], losses[-1], norms[0], norms[-1]))
    batch = block.forward(x)[:32].float()
    single = serve(block, x[:32]).float()
    torch.cuda.synchronize()
    print("one token at a time against the batch: largest difference %.3g of %.3g" %
          (float((single - batch).abs().max()), float(batch.abs().max())))
    if not losses[-1] < 0.9 * losses[0]:
        raise SystemExit("the loss did not fall")


if __name__ == "__main__":
    main()
