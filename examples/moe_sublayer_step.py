"""Trains one mixture-of-experts sublayer for a few steps with the library's
training operators and its optimizer steps.

    python examples/moe_sublayer_step.py [--tokens 4096] [--steps 20]

A step: layer norm, its output kept for the backward pass in 8 bits; routing
of each token to topk experts, with the balance loss; the experts' products;
the mean squared error against a fixed target. Back: the experts' weight
gradients from the checkpoint, the router's and the norm's backward passes;
then Muon on the matrices and AdamW on the norm's weight and bias.

The norm's output itself is not kept: what the backward pass needs of it comes
from the checkpoint (its weight gradients) or from the norm's input (its own
gradient). The experts' matrix products are torch's.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import muon_newton_schulz_03_amd as mu  # noqa: E402


class MoeSublayer:
    """Weights, optimizer state and buffers of a sublayer of `tokens` tokens a step."""

    def __init__(self, tokens, width, out, experts, topk, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        bf, f32 = torch.bfloat16, torch.float32

        def randn(*shape, scale=1.0):
            return torch.randn(shape, generator=g, device="cuda").mul_(scale)

        self.topk = topk
        # the experts' matrices and gradients lie side by side; the optimizer takes them one by one
        self.experts = randn(experts, out, width, scale=width ** -0.5).to(bf)
        self.router = randn(experts, width, scale=width ** -0.5).to(bf)
        self.norm = [torch.ones((1, width), dtype=bf, device="cuda"), torch.zeros((1, width), dtype=bf, device="cuda")]
        self.moms = [torch.zeros_like(w) for w in self.matrices()]
        self.adam = [[torch.zeros((1, width), device="cuda") for _ in range(2)] for _ in range(2)]
        self.steps = 0
        # what a step writes, made once
        i32 = dict(dtype=torch.int32, device="cuda")
        self.y = torch.empty((tokens, width), dtype=bf, device="cuda")
        self.ckpt = mu.Checkpoint.empty(tokens, width)
        self.mean, self.rstd = torch.empty(tokens, device="cuda"), torch.empty(tokens, device="cuda")
        self.choice = torch.empty((tokens, topk), **i32)
        self.share = torch.empty((tokens, topk), device="cuda")
        self.counts, self.offsets = torch.empty(experts + 1, **i32), torch.empty(experts + 1, **i32)
        self.rows = torch.empty(tokens * topk, **i32)
        self.balance = torch.empty(1, device="cuda")
        self.dexperts = torch.empty_like(self.experts)
        self.drouter = torch.empty((1, experts, width), dtype=bf, device="cuda")
        self.dlogits = torch.empty((tokens, experts), dtype=f32, device="cuda")
        self.dnorm = [torch.empty_like(w) for w in self.norm]
        self.dx = torch.empty((tokens, width), dtype=bf, device="cuda")

    def matrices(self):
        return [*self.experts.unbind(0), self.router]

    def step(self, x, target, lr=2e-2, norm_lr=2e-3):
        """One training step on x (tokens x width, bf16); returns (error, balance loss, expert counts)."""
        # forward
        mu.muon_layernorm_forward(x, self.y, self.mean, self.rstd, *self.norm, ckpt=self.ckpt)
        logits = (self.y @ self.router.t()).float()
        mu.muon_route_forward(logits, self.choice, self.share, self.counts, self.offsets, self.rows, self.balance)
        ends = self.offsets.tolist()
        rows = self.rows[:ends[-1]].long()       # the slots in expert order
        token = torch.div(rows, self.topk, rounding_mode="floor")
        inputs = self.y[token]
        hidden = torch.empty((len(rows), self.experts.shape[1]), dtype=torch.bfloat16, device="cuda")
        for e, w in enumerate(self.experts):
            torch.mm(inputs[ends[e]:ends[e + 1]], w.t(), out=hidden[ends[e]:ends[e + 1]])
        share = self.share.view(-1)[rows]
        z = torch.zeros(target.shape, device="cuda").index_add_(0, token, hidden.float() * share[:, None])
        diff = z - target
        error = diff.square().mean()

        # backward
        dz = (diff * (2 / diff.numel()))[token]
        dshare = torch.zeros(self.share.numel(), device="cuda")
        dshare[rows] = (dz * hidden.float()).sum(1)
        dhidden = (dz * share[:, None]).to(torch.bfloat16)
        mu.muon_ckpt_weight_grad(dhidden, self.ckpt, self.dexperts, self.offsets, self.rows[:len(rows)], self.topk)
        mu.muon_route_backward(logits, self.choice, self.counts, self.dlogits, dweights=dshare.view_as(self.share),
                               dloss=torch.ones(1, device="cuda"))
        dlogits = self.dlogits.to(torch.bfloat16)
        mu.muon_ckpt_weight_grad(dlogits, self.ckpt, self.drouter)
        dy = (dlogits @ self.router).float()
        for e, w in enumerate(self.experts):
            if ends[e + 1] > ends[e]:
                dy.index_add_(0, token[ends[e]:ends[e + 1]], (dhidden[ends[e]:ends[e + 1]] @ w).float())
        mu.muon_layernorm_backward(dy.to(torch.bfloat16), x, self.mean, self.rstd, self.dx, self.norm[0], *self.dnorm)

        # update
        self.steps += 1
        mu.muon_step(self.matrices(), [*self.dexperts.unbind(0), self.drouter[0]], self.moms, lr=lr)
        mu.muon_adamw_step(self.norm, self.dnorm, *self.adam, lr=norm_lr, step=self.steps)
        return error, self.balance.clone(), self.counts


def main(tokens=4096, width=512, out=256, experts=16, topk=4, steps=20, quiet=False):
    layer = MoeSublayer(tokens, width, out, experts, topk)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    teacher = torch.randn((width, out), generator=g, device="cuda") * width ** -0.5
    errors = []
    for i in range(steps):
        x = torch.randn((tokens, width), generator=g, device="cuda").to(torch.bfloat16)
        error, balance, counts = layer.step(x, torch.tanh(x.float() @ teacher))
        errors.append(float(error))
        if not quiet:
            c = counts[:experts]
            print(f"step {i + 1:3d}  error {errors[-1]:.4f}  balance loss {float(balance):.4f}  "
                  f"slots per expert {int(c.min())}..{int(c.max())}", flush=True)
    return errors


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, value in (("tokens", 4096), ("width", 512), ("out", 256), ("experts", 16), ("topk", 4), ("steps", 20)):
        ap.add_argument("--" + name, type=int, default=value)
    main(**vars(ap.parse_args()))
