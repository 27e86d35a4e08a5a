"""The feed-forward half of a block on one GPU: y = x + routed(n) + shared(n),
n = layer_norm(x), with routed experts (top-k, weights renormalised) and one
dense gated feed-forward block beside them.

Trains the block for a few steps on a seeded synthetic target (autograd through
layer_norm, moe_layer and gated_ffn), then quantizes both kinds of experts to
4 bits and decodes token by token with them, as a server would.

MixedBlock is a whole block: two projections (bias, activation) mix the features,
the joint norms and gates what they give, adds it to the residual stream and
norms the stream for the experts.  It decodes with the bf16 weights it was trained
with, the expert layer in two kernels.

    python examples/moe_block.py [--tokens 512 --hidden 256 --inter 128 --experts 8 --topk 2 --steps 20]

Needs a GB300 and the built library
(python -c "import __graft_entry__ as g; g.build()").
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from routed_grouped_gemm_routing_gb300.block import (  # noqa: E402
    FFNWorkspace, W4Experts, W4Linear, gated_ffn, layer_norm, layer_norm_forward, linear, quantize_w4, residual_norm)
from routed_grouped_gemm_routing_gb300.layer import DecodeLayer, MoEWorkspace, moe_layer  # noqa: E402

BF = torch.bfloat16


class MoEBlock:
    """Parameters of one block and its training form."""

    def __init__(self, H: int, I: int, E: int, k: int, seed: int = 0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)

        def p(*shape, std):
            return (torch.randn(shape, generator=g, device=device) * std).to(BF).requires_grad_()

        self.H, self.I, self.E, self.k = H, I, E, k
        self.norm_w = torch.ones(H, device=device, requires_grad=True)
        self.norm_b = torch.zeros(H, device=device, requires_grad=True)
        self.router = p(H, E, std=H ** -0.5)
        self.W1, self.W2 = p(E, H, 2 * I, std=H ** -0.5), p(E, I, H, std=I ** -0.5)
        self.S1, self.S2 = p(H, 2 * I, std=H ** -0.5), p(I, H, std=I ** -0.5)
        self._ws = {}

    def parameters(self):
        return [self.norm_w, self.norm_b, self.router, self.W1, self.W2, self.S1, self.S2]

    def workspaces(self, T: int):
        """The routed and the dense experts' buffers for T tokens, kept from step to step."""
        if T not in self._ws:
            self._ws[T] = (MoEWorkspace(T, self.H, self.I, self.E, self.k), FFNWorkspace(T, self.H, self.I))
        return self._ws[T]

    def route(self, n):
        w, idx = torch.topk((n @ self.router).float(), self.k, dim=1)
        return idx.to(torch.int32), torch.softmax(w, dim=1)

    def __call__(self, x):
        """y bf16 [T, H] for x bf16 [T, H]."""
        routed_ws, shared_ws = self.workspaces(x.shape[0])
        n = layer_norm(x, self.norm_w, self.norm_b)
        idx, w = self.route(n)
        return x + moe_layer(n, self.W1, self.W2, idx, w, workspace=routed_ws) + gated_ffn(n, self.S1, self.S2, shared_ws)


class W4Block:
    """The same block for decoding, experts in 4 bits."""

    def __init__(self, b: MoEBlock, group: int = 128):
        with torch.no_grad():
            self.norm_w, self.norm_b, self.k = b.norm_w.detach(), b.norm_b.detach(), b.k
            # the router stays as it is: its decisions are worth more than its bytes
            self.router = b.router.detach()
            self.routed = W4Experts.quantize(b.W1.detach(), b.W2.detach(), group)
            self.shared = W4Experts.quantize(b.S1.detach(), b.S2.detach(), group)

    def __call__(self, x):
        n, _, _ = layer_norm_forward(x, self.norm_w, self.norm_b)
        w, idx = torch.topk((n @ self.router).float(), self.k, dim=1)
        return x + self.routed(n, idx.to(torch.int32), torch.softmax(w, dim=1)) + self.shared(n)


class MixedBlock(MoEBlock):
    """A block whose first half is two projections:
    s = x + gate norm(m) with m = gelu(x P1 + b1) P2 + b2,   y = s + routed(n) + shared(n), n = norm(s)."""

    def __init__(self, H: int, I: int, E: int, k: int, seed: int = 0, device="cuda"):
        super().__init__(H, I, E, k, seed, device)
        g = torch.Generator(device=device).manual_seed(seed + 1)

        def p(*shape, std):
            return (torch.randn(shape, generator=g, device=device) * std).to(BF).requires_grad_()

        self.P1, self.P2 = p(H, 2 * H, std=H ** -0.5), p(2 * H, H, std=(2 * H) ** -0.5)
        self.b1, self.b2 = p(2 * H, std=0.1), p(H, std=0.1)
        self.post_w = torch.ones(H, device=device, requires_grad=True)
        self.gate = torch.full((H,), 0.5, device=device, requires_grad=True)

    def parameters(self):
        return super().parameters() + [self.P1, self.P2, self.b1, self.b2, self.post_w, self.gate]

    def first_half(self, x):
        """(s, n) bf16 [T, H]."""
        m = linear(linear(x, self.P1, self.b1, activation="gelu"), self.P2, self.b2)
        return residual_norm(m, x, self.norm_w, self.norm_b, post_weight=self.post_w, gate=self.gate, kind="rms")

    def __call__(self, x, routing=None):
        routed_ws, shared_ws = self.workspaces(x.shape[0])
        s, n = self.first_half(x)
        idx, w = self.route(n) if routing is None else routing
        return s + moe_layer(n, self.W1, self.W2, idx, w, workspace=routed_ws) + gated_ffn(n, self.S1, self.S2, shared_ws)

    def decoder(self):
        """x bf16 [T, H] -> y for a few tokens at a time, on the weights as they are."""
        experts = DecodeLayer(self.router, self.W1, self.W2, self.k, self.S1, self.S2)

        def decode(x):
            with torch.no_grad():
                s, n = self.first_half(x)
                return s + experts(n)

        return decode


def train(block: MoEBlock, tokens: int, steps: int, lr: float = 0.02):
    """Losses of plain gradient steps toward a fixed synthetic target."""
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(tokens, block.H, generator=g, device="cuda").to(BF)
    target = torch.tanh(x.float() @ (torch.randn(block.H, block.H, generator=g, device="cuda") * block.H ** -0.5))
    losses = []
    for _ in range(steps):
        loss = (block(x).float() - target).square().mean()
        loss.backward()
        with torch.no_grad():
            for p in block.parameters():
                p -= (lr * p.grad.float() * (p.float().norm() / p.grad.float().norm().clamp_min(1e-12))).to(p.dtype)
                p.grad = None
        losses.append(loss.detach())
    return x, [float(v) for v in losses]


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    for n, v in (("tokens", 512), ("hidden", 256), ("inter", 128), ("experts", 8), ("topk", 2), ("steps", 20)):
        ap.add_argument(f"--{n}", type=int, default=v)
    a = ap.parse_args()
    block = MoEBlock(a.hidden, a.inter, a.experts, a.topk)
    x, losses = train(block, a.tokens, a.steps)
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f} over {len(losses)} steps")
    decode = W4Block(block)
    with torch.no_grad():
        want = block(x).float()
        got = torch.cat([decode(x[t: t + 1]) for t in range(16)]).float()  # token by token
        rel = float((got - want[:16]).norm() / (want[:16] - x[:16].float()).norm())
    print(f"4-bit decoding, one token at a time: {rel:.3f} of the block's update off its bf16 form")
    head = W4Linear(*quantize_w4(torch.randn(a.hidden, 1000, device="cuda").to(BF), 32), 32)
    print(f"logits of one token through a 4-bit projection: {list(head(got[:1].to(BF)).shape)}")
    mixed = MixedBlock(a.hidden, a.inter, a.experts, a.topk)
    x, losses = train(mixed, a.tokens, a.steps)
    print(f"mixed block: loss {losses[0]:.4f} -> {losses[-1]:.4f} over {len(losses)} steps")
    decode = mixed.decoder()
    with torch.no_grad():
        want = mixed(x).float()
    got = torch.cat([decode(x[t: t + 1]) for t in range(16)]).float()
    rel = float((got - want[:16]).norm() / want[:16].norm())
    print(f"bf16 decoding, one token at a time: {rel:.4f} off the training form")


if __name__ == "__main__":
    main()
