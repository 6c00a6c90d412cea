"""The mixture-of-experts example: its gradients against torch's autograd of
the same sublayer in float32 on the CPU, and a falling error over a few steps."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_gradients_of_one_step(gpu_lib):
    import moe_sublayer_step as ex
    tokens, width, out, experts, topk = 96, 128, 64, 8, 2
    layer = ex.MoeSublayer(tokens, width, out, experts, topk)
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    x = torch.randn((tokens, width), generator=g, device="cuda").to(torch.bfloat16)
    target = torch.randn((tokens, out), generator=g, device="cuda")
    leaves = [t.float().cpu().requires_grad_() for t in (x, layer.experts, layer.router, *layer.norm)]
    error, balance, counts = layer.step(x, target)
    xl, we, wr, gain, shift = leaves
    y = torch.nn.functional.layer_norm(xl, (width,), gain[0], shift[0])
    # the checkpoint's values stand for y where the weights' gradients read it: same gradients up to its rounding
    p = torch.softmax(y @ wr.t(), 1)
    idx = layer.choice.long().cpu()
    w = torch.gather(p, 1, idx)
    w = w / w.sum(1, keepdim=True)
    z = (torch.stack([y @ e.t() for e in we], 1)[torch.arange(tokens)[:, None], idx] * w[:, :, None]).sum(1)
    n = counts[:experts].float().cpu()
    loss = (z - target.cpu()).square().mean() + 1e-2 * experts / (topk * tokens) * (n * p.sum(0) / tokens).sum()
    loss.backward()
    assert abs(float(error + balance[0]) - loss.item()) <= 2e-2 * loss.item()
    # bf16 values through three products (2^-8 each way) and e4m3 checkpoints (2^-4 a value, averaged over the tokens)
    for name, got, ref, tol in (("dx", layer.dx, xl.grad, 3e-2), ("experts", layer.dexperts, we.grad, 2.0 ** -4),
                                ("gain", layer.dnorm[0][0], gain.grad[0], 3e-2),
                                ("shift", layer.dnorm[1][0], shift.grad[0], 3e-2)):
        got = got.float().cpu()
        rel = float((got - ref).norm() / ref.norm())
        assert rel <= tol, (name, rel)


def test_error_falls(gpu_lib):
    import moe_sublayer_step as ex
    errors = ex.main(tokens=1024, width=256, out=128, experts=8, topk=2, steps=12, quiet=True)
    assert errors[-1] < 0.8 * errors[0], errors


def test_router_gradient_of_one_step(gpu_lib):
    """The router's weight gradient, which takes the balance loss, the gate weights and the checkpoint together."""
    import moe_sublayer_step as ex
    tokens, width, out, experts, topk = 192, 128, 64, 8, 3
    layer = ex.MoeSublayer(tokens, width, out, experts, topk, seed=5)
    g = torch.Generator(device="cuda")
    g.manual_seed(6)
    x = torch.randn((tokens, width), generator=g, device="cuda").to(torch.bfloat16)
    target = torch.randn((tokens, out), generator=g, device="cuda")
    xl, we, gain, shift = [t.float().cpu() for t in (x, layer.experts, *layer.norm)]
    router = layer.router.float().cpu().requires_grad_()
    _, _, counts = layer.step(x, target)
    y = torch.nn.functional.layer_norm(xl, (width,), gain[0], shift[0])
    p = torch.softmax(y @ router.t(), 1)
    idx = layer.choice.long().cpu()
    w = torch.gather(p, 1, idx)
    w = w / w.sum(1, keepdim=True)
    z = (torch.stack([y @ e.t() for e in we], 1)[torch.arange(tokens)[:, None], idx] * w[:, :, None]).sum(1)
    n = counts[:experts].float().cpu()
    loss = (z - target.cpu()).square().mean() + 1e-2 * experts / (topk * tokens) * (n * p.sum(0) / tokens).sum()
    loss.backward()
    # e4m3 checkpoints, 2^-4 a value, as for the experts
    rel = float((layer.drouter[0].float().cpu() - router.grad).norm() / router.grad.norm())
    assert rel <= 2.0 ** -4, rel
