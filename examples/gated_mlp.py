"""A gated MLP, y = down(silu(gate(x)) * up(x)), trained and then called for one
token, on the low-bit linear layer's kernels:

    forward    x, h quantised to MXFP4 for the products; x, h, gate(x) and up(x)
               kept in 8 bits, the only activations that the backward pass reads
    backward   dh, dgate, dup and dx in bfloat16, dW in float32 added up over the
               micro-batches of a step
    weights    float32 masters, quantised into the layers after each step

The target is another random MLP of the same shape, so that there is a loss to
bring down. Nothing is downloaded; all data is synthetic.

    python examples/gated_mlp.py [--width 1024] [--hidden 2048] [--tokens 512] [--steps 60]
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from bit_quantization_block_amd import lq  # noqa: E402


class GatedMlp:
    """`masters`: float32 (gate, up, down) weights; `tokens`: the most rows of a call; `fmt`: of the 8-bit checkpoints."""

    def __init__(self, masters, tokens: int, fmt: str = "int8"):
        self.masters = masters
        hidden, width = masters[0].shape
        self.gate, self.up, self.down = (lq.Mx4Linear(w, rows=tokens) for w in masters)
        self.x8 = lq.Ckpt8(tokens, width, fmt)
        self.h8 = lq.Ckpt8(tokens, hidden, fmt)
        self.act = lq.SwigluCkpt8(tokens, hidden, fmt=fmt)
        self.grads = [torch.zeros_like(w) for w in masters]

    def forward(self, x):
        """y for as many rows as the checkpoints have, which receive what backward() needs."""
        h = self.act.forward(self.gate.forward(x, ckpt=self.x8), self.up.forward(x))
        return self.down.forward(h, ckpt=self.h8)

    def backward(self, dy):
        """dx; the weights' gradients are added to self.grads."""
        self._add(2, self.down, dy, self.h8)
        dgate, dup = self.act.backward(self.down.dgrad(dy))
        self._add(0, self.gate, dgate, self.x8)
        self._add(1, self.up, dup, self.x8)
        return self.gate.dgrad(dgate) + self.up.dgrad(dup)

    def _add(self, i, layer, dy, kept):
        layer.wgrad(dy, kept, dw_in=self.grads[i], out=self.grads[i])

    def step(self, rate):
        """Plain gradient descent on the masters, whose quantised form the layers then hold."""
        for w, g, layer in zip(self.masters, self.grads, (self.gate, self.up, self.down)):
            w.sub_(g, alpha=rate)
            layer.load(w)
            g.zero_()

    def call(self, x, act):
        """y for any number of rows, which leaves what forward() kept as it is; `act` is a SwigluCkpt8 of that many rows,
        whose own checkpoints it fills."""
        return self.down.forward(act.forward(self.gate.forward(x), self.up.forward(x)))


def weights(width, hidden, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    shapes = ((hidden, width), (hidden, width), (width, hidden))
    return [torch.randn(s, generator=gen, device="cuda") * s[1] ** -0.5 for s in shapes]


def plain(masters, x):
    g, u = x @ masters[0].t(), x @ masters[1].t()
    return (torch.nn.functional.silu(g) * u) @ masters[2].t()


def train(width, hidden, tokens, steps, micro_batches=2, rate=None, fmt="int8", say=print):
    """The losses of the steps, and the trained MLP."""
    target = weights(width, hidden, 1)
    # start near the target: its weights and as much noise again as half of them
    mlp = GatedMlp([t + 0.5 * w for t, w in zip(target, weights(width, hidden, 2))], tokens, fmt)
    rate = 0.2 * width ** 0.5 if rate is None else rate
    gen = torch.Generator(device="cuda").manual_seed(3)
    losses = []
    for i in range(steps):
        total = torch.zeros((), device="cuda")
        for _ in range(micro_batches):
            x = torch.randn(tokens, width, generator=gen, device="cuda").bfloat16()
            off = mlp.forward(x).float() - plain(target, x.float())
            total += off.square().mean() / micro_batches
            mlp.backward((2 * off / (off.numel() * micro_batches)).bfloat16())
        mlp.step(rate)
        losses.append(total.item())
        if i % 10 == 0 or i == steps - 1:
            say(f"step {i}: loss {losses[-1]:.4f}", flush=True)
    return losses, mlp


def main():
    a = argparse.ArgumentParser()
    a.add_argument("--width", type=int, default=1024)
    a.add_argument("--hidden", type=int, default=2048)
    a.add_argument("--tokens", type=int, default=512)
    a.add_argument("--steps", type=int, default=60)
    a.add_argument("--fmt", choices=("int8", "e4m3"), default="int8")
    a = a.parse_args()
    losses, mlp = train(a.width, a.hidden, a.tokens, a.steps, fmt=a.fmt)
    kept = sum(c.codes.numel() + c.scales.numel() for c in (mlp.x8, mlp.h8, mlp.act.gate, mlp.act.up))
    wide = 2 * a.tokens * (a.width + 3 * a.hidden)
    print(f"kept for the backward pass: {kept / 1e6:.2f} MB (bfloat16: {wide / 1e6:.2f} MB)")
    act = lq.SwigluCkpt8(1, a.hidden, fmt=a.fmt)
    x = torch.randn(1, a.width, device="cuda").bfloat16()
    for _ in range(10):
        mlp.call(x, act)
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(100):
        mlp.call(x, act)
    torch.cuda.synchronize()
    print(f"one token: {(time.perf_counter() - t) * 1e4:.1f} us a call")


if __name__ == "__main__":
    main()
