"""The feed-forward half of a transformer layer: trained in BF16, then answering from packed 4-bit weights.

    python examples/feed_forward.py

One layer is fitted to the outputs of another with weights near its own.  A training
step runs layer_norm, gated (saving what its backward pass needs), the down
projection, gated_backward and layer_norm_backward; the weights' FP32 copies
are then moved against their gradients.  Afterwards the three matrices are
quantized to NVFP4 and a few tokens answered with packed_gated and packed_gemv.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import int_quantization_amd as iq  # noqa: E402

BF16 = torch.bfloat16


class FeedForward:
    """y = x + down(act(gate(norm(x))) * up(norm(x))); FP32 parameters, BF16 products."""

    def __init__(self, cols, features, act="silu", seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, scale):
            return torch.randn(*shape, generator=gen, device="cuda") * scale

        self.act = act
        self.weight, self.bias = torch.ones(cols, device="cuda"), torch.zeros(cols, device="cuda")
        self.gate, self.up = normal(features, cols, scale=cols ** -0.5), normal(features, cols, scale=cols ** -0.5)
        self.down = normal(cols, features, scale=features ** -0.5)

    def forward(self, x):
        """Output, and what backward needs."""
        n, mean, rstd = iq.layer_norm(x, self.weight, self.bias)
        gate, up, down = self.gate.to(BF16), self.up.to(BF16), self.down.to(BF16)
        h, saved = iq.gated(n, gate, up, self.act, save=True)
        return x + h @ down.t(), (x, n, mean, rstd, gate, up, down, h, saved)

    def backward(self, dy, kept):
        """Gradients of the input and of the parameters, from the output's."""
        x, n, mean, rstd, gate, up, down, h, saved = kept
        ddown = dy.t() @ h
        dn, dgate, dup = iq.gated_backward(dy @ down, n, gate, up, saved, self.act)
        dx, dweight, dbias = iq.layer_norm_backward(dn, x, self.weight, mean, rstd)
        return dy + dx, (dweight, dbias, dgate, dup, ddown)

    def step(self, grads, rate):
        for p, g in zip((self.weight, self.bias, self.gate, self.up, self.down), grads):
            p -= rate * g.float()

    def packed(self, fmt="nvfp4"):
        """The three matrices in 4 bits."""
        return [iq.quantize(w.to(BF16), fmt, "block", stats=False) for w in (self.gate, self.up, self.down)]

    def answer(self, x, packed):
        """The output for up to 64 tokens from packed weights."""
        gate, up, down = packed
        n = iq.layer_norm(x, self.weight, self.bias)[0]
        return x + iq.packed_gemv(down, iq.packed_gated(gate, up, n, self.act))


def train(cols=512, features=1408, tokens=1024, steps=30, rate=0.1, seed=1):
    """Fits a layer to another's outputs; the fitted layer and the loss of every step."""
    teacher, layer, other = (FeedForward(cols, features, seed=s) for s in (seed, seed, seed + 1))
    for name in ("gate", "up", "down"):
        setattr(layer, name, getattr(teacher, name) + 0.3 * getattr(other, name))
    gen = torch.Generator(device="cuda").manual_seed(seed + 2)
    losses = []
    for _ in range(steps):
        x = torch.randn(tokens, cols, generator=gen, device="cuda").to(BF16)
        y, kept = layer.forward(x)
        off = (y - teacher.forward(x)[0]).float()
        losses.append((off * off).mean())
        layer.step(layer.backward((off * (2 / tokens)).to(BF16), kept)[1], rate)
    return layer, torch.stack(losses).tolist()


def main():
    layer, losses = train()
    for i in range(0, len(losses), 5):
        print(f"step {i:3d}  loss {losses[i]:.4f}")
    x = torch.randn(4, layer.weight.numel(), device="cuda").to(BF16)
    full, few = layer.forward(x)[0].float(), layer.answer(x, layer.packed()).float()
    print(f"4 tokens from packed weights: off by {((few - full).norm() / full.norm()).item():.3f} of the BF16 answer")


if __name__ == "__main__":
    main()
