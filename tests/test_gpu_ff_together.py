"""The feed-forward operators together: a whole expert sublayer against
autograd in 64 bits, gradients against differences, captured and replayed, on
other streams, in buffers past 32 bits, and twice over for the same bits."""
import os
import sys

import numpy as np
import pytest
import torch

from oracle import ff_oracle as F
from test_gpu_ff_ops import BF, F32, HALF, KEY, MARK, U, gen, grouped64, key_of, lists, mat, near, out_mat, randn, stack

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def buffers(mu, tokens, topk, experts, n, k, dtype):
    """What a sublayer's pass writes."""
    slots = tokens * topk
    new = lambda rows, cols, dt=dtype: torch.full((rows, cols), MARK, device="cuda").to(dt)  # noqa: E731
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    return dict(idx=i32(tokens, topk), w=torch.zeros((tokens, topk), device="cuda"), counts=i32(experts + 1), offsets=i32(experts + 1),
                rows=i32(slots), loss=torch.zeros(1, device="cuda"), h=new(slots, n), gate=new(slots, n), up=new(slots, n),
                z=new(slots, k), y=new(tokens, k), dz=new(slots, k), dw=torch.zeros((tokens, topk), device="cuda"),
                dh=new(slots, n), dgate=new(slots, n), dup=new(slots, n), dxs=new(slots, k), dx=new(tokens, k))


def sublayer(mu, v, x, logits, wg, wu, wd, dy, key, p):
    """Routing, experts, sum, and back to the gradient of x (the residual's included)."""
    topk = v["idx"].shape[1]
    mu.muon_route_forward(logits, v["idx"], v["w"], v["counts"], v["offsets"], v["rows"], v["loss"])
    lists_ = dict(offsets=v["offsets"], rows=v["rows"])
    mu.muon_gated_forward(x, wg, wu, v["h"], v["gate"], v["up"], rows_per_token=topk, **lists_)
    mu.muon_expert_forward(v["h"], wd, v["z"], scatter=True, **lists_)
    mu.muon_combine_forward(v["z"], v["y"], v["w"], v["idx"], residual=x, p=p, key=key)
    mu.muon_combine_backward(dy, v["z"], v["dz"], v["dw"], v["w"], v["idx"], v["rows"], p=p, key=key)
    mu.muon_expert_backward(v["dz"], wd, v["dh"], v["offsets"])
    mu.muon_gated_backward(v["dh"], v["gate"], v["up"], wg, wu, v["dgate"], v["dup"], v["dxs"], **lists_)
    mu.muon_combine_forward(v["dxs"], v["dx"], indices=v["idx"], residual=dy)


def inputs(g, tokens, topk, experts, n, k, dtype, masked=0):
    logits = randn(g, tokens, experts)
    if masked:
        logits[-masked:] = -float("inf")
    x, dy = randn(g, tokens, k).to(dtype), randn(g, tokens, k).to(dtype)
    return (x, logits, randn(g, experts, n, k, scale=k ** -0.5).to(dtype), randn(g, experts, n, k, scale=k ** -0.5).to(dtype),
            randn(g, experts, k, n, scale=n ** -0.5).to(dtype), dy)


@pytest.mark.parametrize("dtype,tol", [(F32, 2e-5), (BF, 2e-2)])
@pytest.mark.parametrize("tokens,topk,experts,n,k,masked", [(200, 2, 8, 96, 64, 13), (65, 3, 5, 33, 47, 1), (1, 4, 16, 128, 128, 0)])
def test_sublayer_against_autograd(gpu_lib, tokens, topk, experts, n, k, masked, dtype, tol):
    """Each result's norm is off by a few roundings of its type: bf16 seven of 2^-9 on average, float32 sums of up to 128."""
    mu, g, p = gpu_lib, gen(tokens), 0.2
    x, logits, wg, wu, wd, dy = inputs(g, tokens, topk, experts, n, k, dtype, masked)
    v = buffers(mu, tokens, topk, experts, n, k, dtype)
    sublayer(mu, v, x, logits, wg, wu, wd, dy, key_of(*KEY), p)
    # the same in 64 bits on the CPU, with the routing's weights and choices as stored
    leaf = lambda t: t.double().cpu().requires_grad_()  # noqa: E731
    xl, gl, ul, dl, wl = leaf(x), leaf(wg), leaf(wu), leaf(wd), leaf(v["w"])
    idx = v["idx"].long().cpu()
    there = idx >= 0
    e = idx.clamp(min=0)
    gate = torch.stack([xl @ m.t() for m in gl], 1)[torch.arange(tokens)[:, None], e]
    up = torch.stack([xl @ m.t() for m in ul], 1)[torch.arange(tokens)[:, None], e]
    h = torch.nn.functional.silu(gate) * up
    z = torch.einsum("tjn,tjkn->tjk", h, dl[e])
    f = torch.from_numpy(F.dropped((tokens, k), p, *KEY))
    y = xl + (z * (wl * there)[:, :, None]).sum(1) * f
    (y * dy.double().cpu()).sum().backward()
    for name, got, ref in (("y", v["y"], y.detach()), ("dx", v["dx"], xl.grad), ("dweights", v["dw"], wl.grad)):
        rel = float((got.double().cpu() - ref).norm() / ref.norm())
        assert rel <= tol, (name, rel)
    assert int(v["counts"][-1]) == tokens - masked


def test_example_runs_and_its_gradients(gpu_lib):
    import gated_sublayer_step as ex
    tokens, width, hidden, experts, topk = 256, 128, 64, 8, 2
    layer = ex.GatedSublayer(tokens, width, hidden, experts, topk, p=0.1)
    g = gen(3)
    x, dout = randn(g, tokens, width).to(BF), randn(g, tokens, width, scale=1e-2).to(BF)
    leaf = lambda t: t.double().cpu().requires_grad_()  # noqa: E731
    xl, gl, ul, dl, rl, gain, shift = [leaf(t) for t in (x, layer.wgate, layer.wup, layer.wdown, layer.router, *layer.norm)]
    seed, offset = layer.key.tolist()
    out = layer.forward(x).double().cpu()
    layer.backward(x, dout)
    y = torch.nn.functional.layer_norm(xl, (width,), gain[0], shift[0])
    probs = torch.softmax(y @ rl.t(), 1)
    e = layer.choice.long().cpu()
    w = torch.gather(probs, 1, e)
    w = w / w.sum(1, keepdim=True)
    t = torch.arange(tokens)[:, None]
    h = torch.nn.functional.silu(torch.stack([y @ m.t() for m in gl], 1)[t, e]) * torch.stack([y @ m.t() for m in ul], 1)[t, e]
    z = torch.einsum("tjn,tjkn->tjk", h, dl[e])
    ref = xl + (z * w[:, :, None]).sum(1) * torch.from_numpy(F.dropped((tokens, width), 0.1, seed, offset))
    n = layer.counts[:experts].double().cpu()
    loss = (ref * dout.double().cpu()).sum() + 1e-2 * experts / (topk * tokens) * (n * probs.sum(0) / tokens).sum()
    loss.backward()
    # bf16 values through up to six products, 2^-9 a rounding on average; e4m3 checkpoints in the weights' gradients, 2^-4 at most a value
    for name, got, want, tol in (("out", out, ref.detach(), 2e-2), ("dx", layer.dx, xl.grad, 3e-2), ("wgate", layer.grads[0], gl.grad, 2.0 ** -4),
                                 ("wup", layer.grads[1], ul.grad, 2.0 ** -4), ("wdown", layer.grads[2], dl.grad, 2.0 ** -4),
                                 ("router", layer.drouter[0], rl.grad, 2.0 ** -4), ("gain", layer.dnorm[0][0], gain.grad[0], 3e-2),
                                 ("shift", layer.dnorm[1][0], shift.grad[0], 3e-2)):
        rel = float((got.double().cpu() - want).norm() / want.norm())
        assert rel <= tol, (name, rel)
    errors = ex.main(tokens=256, width=128, hidden=64, experts=8, topk=2, steps=3, quiet=True)
    assert len(errors) == 3 and all(np.isfinite(errors))


def test_gradients_against_differences(gpu_lib):
    """Central differences of the float32 forward passes along a direction v. With a loss linear in the outputs, sums of the
    outputs' roundings (each below 2^-23 sqrt(K) of the output's size for sums of K random terms, at random) over the step
    stay below; the products are linear in each operand, the activation's third derivative adds step^2 / 6 of its size."""
    mu, g = gpu_lib, gen(31)
    counts, n, k, topk = [30, 0, 51], 40, 56, 2
    slots, tokens = 81, 60
    offsets, rows = lists(g, counts, topk, tokens)
    x, wg, wu, r = randn(g, tokens, k), stack(g, 3, n, k, F32), stack(g, 3, n, k, F32), randn(g, slots, n)
    wd, r2 = stack(g, 3, k, n, F32), randn(g, slots, k)

    def hidden(x, wg, wu, saved=False):
        h, gate, up = (torch.zeros((slots, n), device="cuda") for _ in range(3))
        mu.muon_gated_forward(x, wg, wu, h, gate, up, offsets, rows, topk, "gelu")
        return (h, gate, up) if saved else float((h.double() * r.double()).sum())

    eps = 1e-2
    _, gate, up = hidden(x, wg, wu, True)
    dgate, dup, dxs = torch.zeros_like(r), torch.zeros_like(r), torch.zeros((tokens * topk, k), device="cuda")
    mu.muon_gated_backward(r, gate, up, wg, wu, dgate, dup, dxs, offsets, rows, "gelu")
    dx = torch.zeros((tokens, k), device="cuda")
    mu.muon_combine_forward(dxs, dx)
    v = randn(g, tokens, k)
    want = (hidden(x + eps * v, wg, wu) - hidden(x - eps * v, wg, wu)) / (2 * eps)
    got = float((dx.double() * v.double()).sum())
    size = float((dx.double() * v.double()).abs().sum())
    assert abs(got - want) <= 1e-3 * size, (got, want, size)
    # the second product and the sum over experts: linear
    h = randn(g, slots, n)
    weights = torch.rand((tokens, topk), generator=g, device="cuda")

    def total(h, weights):
        z, y = torch.zeros((tokens * topk, k), device="cuda"), torch.zeros((tokens, k), device="cuda")
        mu.muon_expert_forward(h, wd, z, offsets, rows, scatter=True)
        mu.muon_combine_forward(z, y, weights, p=0.3, key=key_of(*KEY))
        return z, float((y.double() * r2[:tokens].double()).sum())

    z, _ = total(h, weights)
    # dx in rows' order: slots without a group have no place in it
    full = torch.full((tokens * topk,), -1, dtype=torch.int32, device="cuda")
    full[:slots] = rows
    dz, dw, dh = torch.zeros((tokens * topk, k), device="cuda"), torch.zeros((tokens, topk), device="cuda"), torch.zeros((slots, n), device="cuda")
    mu.muon_combine_backward(r2[:tokens].contiguous(), z, dz, dw, weights, None, full, p=0.3, key=key_of(*KEY))
    mu.muon_expert_backward(dz[:slots].contiguous(), wd, dh, offsets)
    vh, vw = randn(g, slots, n), randn(g, tokens, topk)
    for got, want in ((float((dh.double() * vh.double()).sum()), (total(h + vh, weights)[1] - total(h - vh, weights)[1]) / 2),
                      (float((dw.double() * vw.double()).sum()), (total(h, weights + vw)[1] - total(h, weights - vw)[1]) / 2)):
        assert abs(got - want) <= 1e-4 * abs(got) + 1e-3, (got, want)


def test_captured_and_replayed(gpu_lib):
    """Three replays, each with new inputs and another dropout offset, with eager work between them, bit for bit as eager."""
    mu, p = gpu_lib, 0.1
    shape = (300, 4, 16, 96, 128)
    state = list(inputs(gen(40), *shape, BF, 9)) + [key_of(7, 0)]
    eager, captured = buffers(mu, *shape, BF), buffers(mu, *shape, BF)
    sublayer(mu, captured, *state, p)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sublayer(mu, captured, *state, p)
    masks = []
    for i in (1, 2, 3):
        for t, s in zip(state, list(inputs(gen(40 + i), *shape, BF, 3 * i)) + [key_of(7, i)]):
            t.copy_(s)
        for v in (eager, captured):
            for t in v.values():
                t.fill_(1)
        sublayer(mu, eager, *state, p)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for name in eager:
            assert torch.equal(captured[name], eager[name]), (i, name)
        masks.append((eager["y"] == state[0]).float())
    assert not torch.equal(masks[0], masks[1])
    mu.muon_set_stream(None)


def test_on_other_streams_at_once(gpu_lib):
    """Two sublayers on two streams, over and over, as one after the other."""
    mu, p = gpu_lib, 0.1
    shape = (500, 4, 32, 128, 192)
    states = [list(inputs(gen(50 + i), *shape, BF)) + [key_of(i, 3)] for i in range(2)]
    alone = [buffers(mu, *shape, BF) for _ in range(2)]
    for v, s in zip(alone, states):
        sublayer(mu, v, *s, p)
    torch.cuda.synchronize()
    streams, both = [torch.cuda.Stream() for _ in range(2)], [buffers(mu, *shape, BF) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(4):
        for st, v, s in zip(streams, both, states):
            with torch.cuda.stream(st):
                sublayer(mu, v, *s, p)
    torch.cuda.synchronize()
    for a, b in zip(alone, both):
        for name in a:
            assert torch.equal(a[name], b[name]), name


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shape", [(2000, 8, 64, 256, 512), (3, 2, 16, 1024, 2048), (700, 2, 4, 333, 127)])
def test_same_bits_twice(gpu_lib, shape, dtype):
    mu = gpu_lib
    state = list(inputs(gen(60), *shape, dtype, 1)) + [key_of(1, 2)]
    a, b = buffers(mu, *shape, dtype), buffers(mu, *shape, dtype)
    sublayer(mu, a, *state, 0.1)
    for _ in range(3):
        sublayer(mu, b, *state, 0.1)
        for name in a:
            assert torch.equal(a[name], b[name]), name


def test_rows_without_a_group_are_neither_read_nor_written(gpu_lib):
    """NaN in every slot behind the last group, and around the first."""
    mu, g = gpu_lib, gen(70)
    counts, n, k, topk = [100, 3, 0, 60], 96, 64, 2
    slots, tokens = sum(counts) + 40, 110
    offsets, rows = lists(g, counts, topk, tokens, 20, 20)
    rows[:20], rows[-20:] = -1, -1
    own = torch.zeros(slots, dtype=torch.bool, device="cuda")
    own[20:-20] = True
    for dtype in (BF, F32):
        wg, wu = stack(g, 4, n, k, dtype), stack(g, 4, n, k, dtype)
        dh, gate, up = (mat(randn(g, slots, n), dtype) for _ in range(3))
        for t in (dh, gate, up):
            t[~own] = float("nan")
        dgate, dup, dxs = out_mat(slots, n, dtype), out_mat(slots, n, dtype), out_mat(tokens * topk, k, dtype)
        mu.muon_gated_backward(dh, gate, up, wg, wu, dgate, dup, dxs, offsets, rows)
        assert bool(torch.isfinite(dgate).all() and torch.isfinite(dup).all() and torch.isfinite(dxs).all())
        assert bool((dgate[~own] == MARK).all() and (dup[~own] == MARK).all())
        y = out_mat(slots, k, dtype)
        mu.muon_expert_backward(dh, wg, y, offsets)
        assert bool(torch.isfinite(y).all() and (y[~own] == MARK).all())


@pytest.mark.parametrize("groups", [1025, 3000, 65536])
def test_many_groups(gpu_lib, groups):
    """More groups than a streaming workgroup keeps, and than one pass over the offsets counts; most of them empty."""
    mu, g = gpu_lib, gen(groups)
    n, k, slots = 16, 24, 5000
    at = torch.sort(torch.randint(0, slots + 1, (groups - 1,), generator=g, device="cuda")).values
    at = at // 7 * 7
    offsets = torch.cat([at.new_zeros(1), at, at.new_full((1,), slots)]).to(torch.int32)
    w = (randn(g, groups, n, k) * k ** -0.5).to(BF)
    x, y = mat(randn(g, slots, k), BF), out_mat(slots, n, BF)
    mu.muon_expert_forward(x, w, y, offsets)
    group = torch.searchsorted(offsets.long(), torch.arange(slots, device="cuda"), right=True) - 1
    r = torch.bmm(w[group].float(), x.float()[:, :, None])[:, :, 0].double()
    m = torch.bmm(w[group].float().abs(), x.float().abs()[:, :, None])[:, :, 0].double()
    near(y, r, HALF[BF] * r.abs() + 3 * (2 * k + 2) * U * m, "y")


def test_operands_past_32_bits(gpu_lib):
    """Tokens, weights and outputs that lie beyond 2^32 bytes and 2^31 elements from their buffers' starts."""
    mu, g = gpu_lib, gen(80)
    # gathered rows of a 5 GiB matrix, through registers
    tokens, k, n, slots = 1300000, 2048, 72, 400
    x = torch.empty((tokens, k), dtype=BF, device="cuda")
    at = torch.randint(tokens - 200000, tokens, (slots,), generator=g, device="cuda").to(torch.int32)
    at[::2] //= 9
    x[at.long()] = randn(g, slots, k).to(BF)
    w, y = stack(g, 1, n, k, BF), out_mat(slots, n, BF)
    mu.muon_expert_forward(x, w, y, rows=at, gather=1)
    r, m = grouped64(x[at.long()], w, [0, slots], torch.arange(slots, device="cuda"), False)
    near(y, r, HALF[BF] * r.abs() + (2 * k + 2) * U * m, "gathered")
    # scattered to rows of a wide matrix
    out = torch.full((tokens, k), MARK, dtype=BF, device="cuda")
    to = torch.randperm(tokens, generator=g, device="cuda")[:slots].to(torch.int32)
    to[0] = tokens - 1
    to = to.unique()
    h, wd = mat(randn(g, len(to), 40), BF), stack(g, 1, k, 40, BF)
    mu.muon_expert_forward(h, wd, out, rows=to, scatter=True)
    r, m = grouped64(h, wd, [0, len(to)], torch.arange(len(to), device="cuda"), False)
    near(out[to.long()], r, HALF[BF] * r.abs() + 82 * U * m, "scattered")
    assert int((out[:, 0] != MARK).sum()) <= len(to)
    del x, out
    # groups far apart
    far = torch.empty((3, 1 << 30), dtype=BF, device="cuda")
    w3 = far.as_strided((3, 64, 128), (1 << 30, 128, 1))
    w3.copy_(randn(g, 3, 64, 128) * 128 ** -0.5)
    offsets = torch.tensor([0, 300, 310, 700], dtype=torch.int32, device="cuda")
    x, y = mat(randn(g, 700, 128), BF), out_mat(700, 64, BF)
    mu.muon_expert_forward(x, w3, y, offsets)
    r, m = grouped64(x, w3, offsets.tolist(), torch.arange(700, device="cuda"), False)
    near(y, r, HALF[BF] * r.abs() + 258 * U * m, "far groups")


# 2^27 threads in 2^19 workgroups, 32 rows each: grids past 2^20 workgroups are in test_gpu_ff_forms.py.
def test_more_slots_than_one_launch_counts(gpu_lib):
    """Rows past 2^32 threads' worth: the last ones are those of a call on them alone."""
    mu, g = gpu_lib, gen(81)
    rows, cols = (1 << 24) + 37, 8
    x = torch.empty((rows, cols), dtype=BF, device="cuda").normal_(generator=g)
    y, key = torch.empty_like(x), key_of(3, 4)
    mu.muon_dropout_forward(x, y, 0.5, key)
    for lo in (0, 1 << 23, rows - 500):
        want = F.kept(lo * cols, 500 * cols, 0.5, 3, 4).reshape(500, cols)
        assert np.array_equal((y[lo:lo + 500] != 0).cpu().numpy(), want & (x[lo:lo + 500] != 0).cpu().numpy()), lo
    w = (randn(g, 16, cols) * 0.3).to(BF)
    h, gate, up = (torch.empty((rows, 16), dtype=BF, device="cuda") for _ in range(3))
    mu.muon_gated_forward(x, w, w.clone(), h, gate, up)
    dgate, dup = torch.empty_like(h), torch.empty_like(h)
    mu.muon_gated_backward(h, gate, up, None, None, dgate, dup)
    part = slice(rows - 300, rows)
    h2, g2, u2 = (torch.empty((300, 16), dtype=BF, device="cuda") for _ in range(3))
    mu.muon_gated_forward(x[part], w, w.clone(), h2, g2, u2)
    dg2, du2 = torch.empty_like(h2), torch.empty_like(h2)
    mu.muon_gated_backward(h2, g2, u2, None, None, dg2, du2)
    for a, b in ((h, h2), (gate, g2), (dgate, dg2), (dup, du2)):
        assert torch.equal(a[part], b)


def test_binding_checks(gpu_lib):
    mu, g = gpu_lib, gen(90)
    x, w, y = randn(g, 8, 16), randn(g, 2, 24, 16), torch.empty((8, 24), device="cuda")
    off = torch.tensor([0, 3, 8], dtype=torch.int32, device="cuda")
    mu.muon_expert_forward(x, w, y, off)
    with pytest.raises(ValueError, match="offsets"):
        mu.muon_expert_forward(x, w, y)
    with pytest.raises(ValueError, match="offsets"):
        mu.muon_expert_forward(x, w, y, off[:2])
    with pytest.raises(TypeError, match="offsets"):
        mu.muon_expert_forward(x, w, y, off.long())
    with pytest.raises(ValueError, match="rows"):
        mu.muon_expert_forward(x, w, y, off, torch.zeros(7, dtype=torch.int32, device="cuda"), scatter=True)
    with pytest.raises(mu.MuonError):
        mu.muon_expert_forward(x, w, y, off, scatter=True)
    with pytest.raises(ValueError, match="unit column stride"):
        mu.muon_expert_forward(x, w.transpose(1, 2), y, off)
    with pytest.raises(ValueError, match="activation"):
        mu.muon_gated_forward(x, w, w.clone(), y, offsets=off, activation="tanh")
    with pytest.raises(ValueError, match="groups"):
        mu.muon_gated_forward(x, w, w[:1].clone(), y, offsets=off)
    with pytest.raises(mu.MuonError):
        mu.muon_dropout_forward(x, torch.empty_like(x), 0.5)
    with pytest.raises(TypeError, match="key"):
        mu.muon_dropout_forward(x, torch.empty_like(x), 0.5, torch.zeros(2, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError, match="both are needed"):
        mu.muon_gated_backward(y, y, y, w, None, y.clone(), y.clone())
    with pytest.raises(ValueError, match="rows overlap"):
        mu.muon_expert_forward(x.as_strided((8, 16), (4, 1)), w, y, off)
    for p in (-0.1, 1.0, float("nan")):
        with pytest.raises(mu.MuonError):
            mu.muon_dropout_forward(x, torch.empty_like(x), p, key_of(0, 0))
