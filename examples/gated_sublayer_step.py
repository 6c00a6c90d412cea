"""Trains a gated mixture-of-experts sublayer for a few steps, every product of
the experts and everything around them by the library's operators.

    python examples/gated_sublayer_step.py [--tokens 4096] [--steps 20]

A step: layer norm, its output kept for the backward pass in 8 bits; routing;
the gated block's first half over the slots of each expert, its second product
back to the tokens' order; the sum over a token's experts with dropout and the
residual; the mean squared error against a fixed target. Back through the same
operators; weight gradients from the 8-bit checkpoints of the norm's output and
of the hidden activations; then Muon on the matrices and AdamW on the norm's
weight and bias. Nothing of a step waits for the GPU but the error it prints.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import muon_newton_schulz_03_amd as mu  # noqa: E402


class GatedSublayer:
    """Weights, optimizer state and buffers of a sublayer of `tokens` tokens a step."""

    def __init__(self, tokens, width, hidden, experts, topk, p=0.1, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        bf, f32 = torch.bfloat16, torch.float32

        def randn(*shape, scale=1.0):
            return torch.randn(shape, generator=g, device="cuda").mul_(scale)

        def new(*shape, dtype=bf):
            return torch.empty(shape, dtype=dtype, device="cuda")

        self.topk, self.p = topk, p
        self.wgate = randn(experts, hidden, width, scale=width ** -0.5).to(bf)
        self.wup = randn(experts, hidden, width, scale=width ** -0.5).to(bf)
        self.wdown = randn(experts, width, hidden, scale=hidden ** -0.5).to(bf)
        self.router = randn(experts, width, scale=width ** -0.5).to(bf)
        self.norm = [torch.ones((1, width), dtype=bf, device="cuda"), torch.zeros((1, width), dtype=bf, device="cuda")]
        self.moms = [torch.zeros_like(w) for w in self.matrices()]
        self.adam = [[torch.zeros((1, width), device="cuda") for _ in range(2)] for _ in range(2)]
        self.steps = 0
        self.key = torch.tensor([seed, 0], dtype=torch.int64, device="cuda")  # dropout's seed and offset
        # what a step writes, made once; rows of slots without a token are never read
        slots, i32 = tokens * topk, torch.int32
        self.y, self.ckpt = new(tokens, width), mu.Checkpoint.empty(tokens, width)
        self.mean, self.rstd = new(tokens, dtype=f32), new(tokens, dtype=f32)
        self.choice, self.share = new(tokens, topk, dtype=i32), new(tokens, topk, dtype=f32)
        self.counts, self.offsets, self.rows = new(experts + 1, dtype=i32), new(experts + 1, dtype=i32), new(slots, dtype=i32)
        self.balance = new(1, dtype=f32)
        self.h, self.gate, self.up = new(slots, hidden), new(slots, hidden), new(slots, hidden)
        self.hidden = mu.Checkpoint.empty(slots, hidden)
        self.z, self.out = new(slots, width), new(tokens, width)
        self.dz, self.dshare = new(slots, width), new(tokens, topk, dtype=f32)
        self.dh, self.dgate, self.dup = new(slots, hidden), new(slots, hidden), new(slots, hidden)
        self.dxs, self.dlogits = new(slots, width), new(tokens, experts, dtype=f32)
        self.dy, self.dx, self.dnorm = new(tokens, width), new(tokens, width), [torch.empty_like(w) for w in self.norm]
        self.grads = [torch.empty_like(w) for w in (self.wgate, self.wup, self.wdown)]
        self.drouter = new(1, experts, width)

    def matrices(self):
        return [*self.wgate.unbind(0), *self.wup.unbind(0), *self.wdown.unbind(0), self.router]

    def forward(self, x):
        """The sublayer's output for x (tokens x width, bf16)."""
        mu.muon_layernorm_forward(x, self.y, self.mean, self.rstd, *self.norm, ckpt=self.ckpt)
        self.logits = (self.y @ self.router.t()).float()
        mu.muon_route_forward(self.logits, self.choice, self.share, self.counts, self.offsets, self.rows, self.balance)
        lists = dict(offsets=self.offsets, rows=self.rows)
        mu.muon_gated_forward(self.y, self.wgate, self.wup, self.h, self.gate, self.up, rows_per_token=self.topk, **lists)
        mu.muon_expert_forward(self.h, self.wdown, self.z, scatter=True, **lists)
        mu.muon_ckpt_save(self.h, self.hidden)
        mu.muon_combine_forward(self.z, self.out, self.share, self.choice, residual=x, p=self.p, key=self.key)
        return self.out

    def backward(self, x, dout):
        """All gradients, for dout (tokens x width, bf16) and the balance loss."""
        lists = dict(offsets=self.offsets, rows=self.rows)
        dgate_w, dup_w, ddown_w = self.grads
        mu.muon_combine_backward(dout, self.z, self.dz, self.dshare, self.share, self.choice, self.rows, p=self.p, key=self.key)
        mu.muon_ckpt_weight_grad(self.dz, self.hidden, ddown_w, self.offsets)
        mu.muon_expert_backward(self.dz, self.wdown, self.dh, self.offsets)
        mu.muon_gated_backward(self.dh, self.gate, self.up, self.wgate, self.wup, self.dgate, self.dup, self.dxs, **lists)
        mu.muon_ckpt_weight_grad(self.dgate, self.ckpt, dgate_w, self.offsets, self.rows, self.topk)
        mu.muon_ckpt_weight_grad(self.dup, self.ckpt, dup_w, self.offsets, self.rows, self.topk)
        mu.muon_route_backward(self.logits, self.choice, self.counts, self.dlogits, dweights=self.dshare,
                               dloss=torch.ones(1, device="cuda"))
        dlogits = self.dlogits.to(torch.bfloat16)
        mu.muon_ckpt_weight_grad(dlogits, self.ckpt, self.drouter)
        # the norm's output went to the experts and to the router
        mu.muon_combine_forward(self.dxs, self.dy, indices=self.choice, residual=dlogits @ self.router)
        mu.muon_layernorm_backward(self.dy, x, self.mean, self.rstd, self.dx, self.norm[0], *self.dnorm)
        self.dx += dout  # the residual

    def step(self, x, target, lr=2e-2, norm_lr=2e-3):
        """One training step on x and target (tokens x width); returns (error, balance loss, expert counts)."""
        diff = self.forward(x).float() - target
        error = diff.square().mean()
        self.backward(x, (diff * (2 / diff.numel())).to(torch.bfloat16))
        self.steps += 1
        self.key[1] += 1  # another mask in the next step
        grads = [*(g for w in self.grads for g in w.unbind(0)), self.drouter[0]]
        mu.muon_step(self.matrices(), grads, self.moms, lr=lr)
        mu.muon_adamw_step(self.norm, self.dnorm, *self.adam, lr=norm_lr, step=self.steps)
        return error, self.balance.clone(), self.counts


def main(tokens=4096, width=512, hidden=256, experts=16, topk=4, steps=20, quiet=False):
    layer = GatedSublayer(tokens, width, hidden, experts, topk)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    teacher = torch.randn((width, width), generator=g, device="cuda") * width ** -0.5
    errors = []
    for i in range(steps):
        x = torch.randn((tokens, width), generator=g, device="cuda").to(torch.bfloat16)
        error, balance, counts = layer.step(x, x.float() + torch.tanh(x.float() @ teacher))
        errors.append(float(error))
        if not quiet:
            c = counts[:experts]
            print(f"step {i + 1:3d}  error {errors[-1]:.4f}  balance loss {float(balance):.4f}  "
                  f"slots per expert {int(c.min())}..{int(c.max())}", flush=True)
    return errors


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, value in (("tokens", 4096), ("width", 512), ("hidden", 256), ("experts", 16), ("topk", 4), ("steps", 20)):
        ap.add_argument("--" + name, type=int, default=value)
    main(**vars(ap.parse_args()))
