"""The products' streaming form, long sums that workgroups share, and launches of
more workgroups than a grid's first dimension holds, against 64-bit sums on the
GPU: value by value (as in test_gpu_ff_ops.py) and in norm, where lost precision shows.

That the sizes take the forms meant here is tested on the CPU
(test_product_plan_cpu.py)."""
import numpy as np
import pytest
import torch

from ff_forms import BACKWARD, BOTH, FORWARD, GATED, STREAMING, tight
from oracle import ff_oracle as F
from test_gpu_ff_ops import BF, F32, HALF, KEY, LONG, MARK, U, gen, grouped64, key_of, mat, near, out_mat, randn, stack

pytestmark = pytest.mark.gpu

TYPES = {"bf16": BF, "f32": F32}


def uneven(g, slots, groups):
    """Offsets of groups of any length, some of one tile and less, an empty one, and slots behind the last."""
    share = torch.rand(groups, generator=g, device="cuda") + 0.05
    share[groups // 2] = 0
    ends = (share.cumsum(0) / share.sum() * (slots - 77)).long()
    return torch.cat([ends.new_zeros(1), ends])


def case(g, slots, groups):
    """(offsets, rows, topk): lists, or none for one group. A few entries name no row."""
    if groups == 1:
        return None, None, 1
    rows = torch.randperm(slots, generator=g, device="cuda").to(torch.int32)
    rows[::101] = -1
    return uneven(g, slots, groups).to(torch.int32), rows, 4


def both(got, ref, mag, dtype, terms, what):
    near(got, ref, HALF[dtype] * ref.abs() + (2 * terms + 2) * U * mag, what)
    tight(got, ref, terms, what)


@pytest.mark.parametrize("kind,slots,groups,n,k,dtype,aligned", STREAMING)
def test_streaming_products(gpu_lib, kind, slots, groups, n, k, dtype, aligned):
    mu, g, dtype = gpu_lib, gen(slots + groups + n + k), TYPES[dtype]
    offsets, rows, topk = case(g, slots, groups)
    off = [0, slots] if offsets is None else offsets.tolist()
    lists = dict(offsets=offsets, rows=rows)
    own = torch.arange(slots, device="cuda")
    used = own < off[-1]
    named = used if rows is None else used & (rows >= 0)
    to = own if rows is None else rows.long()
    other = torch.ones(slots, dtype=torch.bool, device="cuda")
    other[to[named]] = False  # rows of a scattered output that no slot names
    if kind == GATED:
        x, w, u = mat(randn(g, -(-slots // topk), k), dtype), stack(g, groups, n, k, dtype), stack(g, groups, n, k, dtype)
        h, gate, up = (out_mat(slots, n, dtype) for _ in range(3))
        mu.muon_gated_forward(x, w, u, h, gate, up, rows_per_token=topk, **lists)
        token = own if rows is None else torch.where(rows < 0, -1, rows // topk).long()
        rg, mg = grouped64(x, w, off, token, False)
        ru, mu_ = grouped64(x, u, off, token, False)
        both(gate[used], rg[used], mg[used], dtype, k, "gate")
        both(up[used], ru[used], mu_[used], dtype, k, "up")
        # the activation takes the float32 products; slopes lie within 1.2 of 0
        e, eu = (2 * k + 2) * U * mg, (2 * k + 2) * U * mu_
        v = rg * torch.sigmoid(rg)
        near(h[used], (v * ru)[used], (HALF[dtype] * (v * ru).abs() + 1.2 * e * (ru.abs() + eu) + v.abs() * eu + 16 * U * (rg * ru).abs())[used], "h")
        for t in (h, gate, up):
            assert bool((t[~used] == MARK).all())
        again = [out_mat(slots, n, dtype) for _ in range(3)]
        mu.muon_gated_forward(x, w, u, *again, rows_per_token=topk, **lists)
        assert all(torch.equal(a, b) for a, b in zip(again, (h, gate, up)))
    elif kind == BOTH:
        dh, gate, up = (mat(randn(g, slots, k), dtype) for _ in range(3))
        w, u = stack(g, groups, k, n, dtype), stack(g, groups, k, n, dtype)
        dgate, dup, dx = out_mat(slots, k, dtype), out_mat(slots, k, dtype), out_mat(slots, n, dtype)
        mu.muon_gated_backward(dh, gate, up, w, u, dgate, dup, dx, **lists)
        a, ma = grouped64(dgate, w, off, own, True)
        b, mb = grouped64(dup, u, off, own, True)
        both(dx[to[named]], (a + b)[named], (ma + mb)[named], dtype, 2 * k, "dx")
        assert bool((dx[other] == MARK).all())
        again = out_mat(slots, n, dtype)
        mu.muon_gated_backward(dh, gate, up, w, u, dgate, dup, again, **lists)
        assert torch.equal(again, dx)
    else:
        back = kind == BACKWARD
        call = mu.muon_expert_backward if back else mu.muon_expert_forward
        x, w = mat(randn(g, slots, k), dtype), stack(g, groups, *((k, n) if back else (n, k)), dtype)
        y = out_mat(slots, n, dtype)
        call(x, w, y, offsets)
        ref, mag = grouped64(x, w, off, own, back)
        both(y[used], ref[used], mag[used], dtype, k, "slot order")
        assert bool((y[~used] == MARK).all())
        if rows is not None:
            z = out_mat(slots, n, dtype)
            call(x, w, z, **lists, scatter=True)
            assert torch.equal(z[to[named]], y[named]) and bool((z[other] == MARK).all())
            # gathered and scattered; a row of x that no entry names is not read
            z = out_mat(slots, n, dtype)
            tokens = mat(randn(g, slots // topk, k), dtype)
            token = torch.where(rows < 0, -1, rows // topk).long()
            call(tokens, w, z, **lists, gather=topk, scatter=True)
            ref, mag = grouped64(tokens, w, off, token, back)
            both(z[to[named]], ref[named], mag[named], dtype, k, "gathered and scattered")
            assert bool((z[other] == MARK).all())


def test_streaming_products_behind_a_captured_graph(gpu_lib):
    """Replays of the streaming forms on new inputs, eager ones between them, bit for bit."""
    mu, g = gpu_lib, gen(5)
    kind, slots, groups, n, k, dtype, _ = next(s for s in STREAMING if s[0] == BOTH and s[2] > 1)
    assert dtype == "bf16"
    offsets, rows, _ = case(g, slots, groups)
    ins = [mat(randn(g, slots, k), BF) for _ in range(3)]
    w, u = stack(g, groups, k, n, BF), stack(g, groups, k, n, BF)
    outs = [[out_mat(slots, c, BF) for c in (k, k, n)] for _ in range(2)]
    step = lambda o: mu.muon_gated_backward(*ins, w, u, *o, offsets=offsets, rows=rows)  # noqa: E731
    step(outs[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(outs[0])
    for _ in range(3):
        for t in ins:
            t.copy_(randn(g, slots, k))
        for t in outs[0] + outs[1]:
            t.fill_(MARK)
        graph.replay()
        step(outs[1])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(*outs))
    mu.muon_set_stream(None)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("fused", [True, False])
@pytest.mark.parametrize("slots,groups,n,k", [(107, 3, 40, 72), (300, 5, 136, 264), (20000, 40, 520, 136), (3, 1, 24, 8200)])
def test_gated_operands_of_one_buffer_and_of_differing_pitches(gpu_lib, slots, groups, n, k, fused, dtype):
    """Both weights as halves of one buffer and the slots' matrices as halves of wide rows, or a pitch of its own for each operand."""
    mu, g = gpu_lib, gen(slots + n + fused)
    offsets = None if groups == 1 else uneven(g, slots, groups).to(torch.int32)
    off, own = [0, slots] if groups == 1 else offsets.tolist(), torch.arange(slots, device="cuda")
    used = own < off[-1]
    if fused:
        w, u = stack(g, groups, 2 * n, k, dtype).split(n, 1)
        halves = [out_mat(slots, 2 * n, dtype) for _ in range(2)]
        (gate, up), (dgate, dup) = (t.split(n, 1) for t in halves)
        x, dh, h, dx = mat(randn(g, slots, k), dtype), mat(randn(g, slots, n), dtype), out_mat(slots, n, dtype), out_mat(slots, k, dtype)
    else:
        w, u = stack(g, groups, n, k, dtype, 16), stack(g, groups, n, k, dtype, 3)
        x, dh = mat(randn(g, slots, k), dtype, 5), mat(randn(g, slots, n), dtype, 8)
        h, gate, up, dgate, dup, dx = (out_mat(slots, c, dtype, e) for c, e in ((n, 1), (n, 8), (n, 0), (n, 16), (n, 24), (k, 7)))
    mu.muon_gated_forward(x, w, u, h, gate, up, offsets)
    mu.muon_gated_backward(dh, gate, up, w, u, dgate, dup, dx, offsets)
    rg, mg = grouped64(x, w, off, own, False)
    ru, mu_ = grouped64(x, u, off, own, False)
    both(gate[used], rg[used], mg[used], dtype, k, "gate")
    both(up[used], ru[used], mu_[used], dtype, k, "up")
    D, G, V = dh.double(), gate.double(), up.double()
    s = torch.sigmoid(G)
    rdg, rdu = D * V * s * (1 + G * (1 - s)), D * G * s
    near(dgate[used], rdg[used], (HALF[dtype] * rdg.abs() + 16 * U * (D * V).abs() * (1 + G.abs()))[used], "dgate")
    near(dup[used], rdu[used], (HALF[dtype] * rdu.abs() + 16 * U * (D * G).abs())[used], "dup")
    a, ma = grouped64(dgate, w, off, own, True)
    b, mb = grouped64(dup, u, off, own, True)
    both(dx[used], (a + b)[used], (ma + mb)[used], dtype, 2 * n, "dx")
    for t in (h, gate, up, dgate, dup, dx):
        assert bool((t[~used] == MARK).all())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("tokens,topk,experts,n,k", LONG)
def test_shared_sums_in_norm(gpu_lib, tokens, topk, experts, n, k, dtype):
    """Long sums whose parts several workgroups make, as exact as float32 sums: parts or operands of fewer bits are not."""
    mu, g, slots = gpu_lib, gen(tokens + n + 2 * k), tokens * topk
    code = mu.MUON_BF16 if dtype == BF else mu.MUON_F32
    ends = torch.arange(experts + 1, device="cuda") * slots // experts
    offsets, off, own = ends.to(torch.int32), ends.tolist(), torch.arange(slots, device="cuda")
    # forward: the gated block's products, and one alone
    assert mu.muon_gated_workspace_size(code, slots, n, k, experts) > 0 and mu.muon_expert_workspace_size(code, slots, n, k, experts) > 0
    x, w, u = mat(randn(g, slots, k), dtype), stack(g, experts, n, k, dtype), stack(g, experts, n, k, dtype)
    h, gate, up, y = (out_mat(slots, n, dtype) for _ in range(4))
    mu.muon_gated_forward(x, w, u, h, gate, up, offsets)
    ref, _ = grouped64(x, w, off, own, False)
    tight(gate, ref, k, "gate")
    tight(up, grouped64(x, u, off, own, False)[0], k, "up")
    mu.muon_expert_forward(x, w, y, offsets)
    tight(y, ref, k, "forward")
    # backward: the sum runs over the weights' rows
    assert mu.muon_gated_workspace_size(code, slots, k, n, experts, 1) > 0 and mu.muon_expert_workspace_size(code, slots, k, n, experts, 1) > 0
    w, u, y = stack(g, experts, k, n, dtype), stack(g, experts, k, n, dtype), out_mat(slots, n, dtype)
    mu.muon_expert_backward(x, w, y, offsets)
    tight(y, grouped64(x, w, off, own, True)[0], k, "backward")
    gate, up = mat(randn(g, slots, k), dtype), mat(randn(g, slots, k), dtype)
    dgate, dup, dx = out_mat(slots, k, dtype), out_mat(slots, k, dtype), out_mat(slots, n, dtype)
    mu.muon_gated_backward(x, gate, up, w, u, dgate, dup, dx, offsets)
    # the gradients' values are no normal ones, but independent with mean near 0: both parts of the sum grow alike
    tight(dx, grouped64(dgate, w, off, own, True)[0] + grouped64(dup, u, off, own, True)[0], 2 * k, "dx")


# ---------------------------------------------------------------------------
# grids past their first dimension's bound of 2^20 workgroups, and the strides behind it
# ---------------------------------------------------------------------------

def test_rows_of_more_than_2_20_workgroups(gpu_lib):
    """A workgroup takes one row of more than 512 columns: the rows behind 2^20 of them are a second turn's. Dropout, the sum
    over experts and its backward pass, the gated block's gradients."""
    mu, g = gpu_lib, gen(91)
    rows, cols, p = (1 << 20) + 37, 520, 0.25
    spans = [slice(0, 5), slice((1 << 20) - 3, (1 << 20) + 5), slice(rows - 5, rows)]
    key, f = key_of(*KEY), {}
    for s in spans:
        f[s.start] = F.kept(s.start * cols, (s.stop - s.start) * cols, p, *KEY).reshape(-1, cols) / (1 - p)
    x = torch.empty((rows, cols), dtype=BF, device="cuda").normal_(generator=g)
    y, dx, dw = torch.full_like(x, MARK), torch.full_like(x, MARK), torch.full((rows, 1), MARK, device="cuda")
    weights = torch.rand((rows, 1), generator=g, device="cuda") + 0.5
    mu.muon_combine_forward(x, y, weights, p=p, key=key)
    dy = torch.empty_like(x).normal_(generator=g)
    mu.muon_combine_backward(dy, x, dx, dw, weights, p=p, key=key)
    for s in spans:
        X, W, D = x[s].double().cpu().numpy(), weights[s].double().cpu().numpy(), dy[s].double().cpu().numpy() * f[s.start]
        for got, ref in ((y[s], X * W * f[s.start]), (dx[s], W * D)):
            assert np.all(np.abs(got.double().cpu().numpy() - ref) <= (HALF[BF] + 4 * U) * np.abs(ref)), s
        # sums of 65 runs of eight products
        assert np.all(np.abs(dw[s].double().cpu().numpy()[:, 0] - (X * D).sum(1)) <= (8 + 16) * U * np.abs(X * D).sum(1)), s
    z = torch.full_like(x, MARK)
    mu.muon_dropout_forward(x, z, p, key, residual=dy)
    for s in spans:
        ref = dy[s].double().cpu().numpy() + x[s].double().cpu().numpy() * f[s.start]
        tol = HALF[BF] * np.abs(ref) + 4 * U * (dy[s].double().abs().cpu().numpy() + np.abs(x[s].double().cpu().numpy() * f[s.start]))
        assert np.all(np.abs(z[s].double().cpu().numpy() - ref) <= tol), s
    assert not bool((y == MARK).all(1).any()) and not bool((dx == MARK).all(1).any()) and not bool((dw == MARK).any())
    del x, y, z, dy, dx
    # a workgroup a row from 1025 columns on
    cols = 1032
    dh, gate, up = (torch.empty((rows, cols), dtype=BF, device="cuda").normal_(generator=g) for _ in range(3))
    dgate, dup = torch.full_like(dh, MARK), torch.full_like(dh, MARK)
    mu.muon_gated_backward(dh, gate, up, None, None, dgate, dup)
    for s in spans:
        part = [torch.empty((s.stop - s.start, cols), dtype=BF, device="cuda") for _ in range(2)]
        mu.muon_gated_backward(dh[s], gate[s], up[s], None, None, *part)
        v, slope = F.act(gate[s].double().cpu().numpy(), "silu")
        D, V = dh[s].double().cpu().numpy(), up[s].double().cpu().numpy()
        assert torch.equal(part[0], dgate[s]) and torch.equal(part[1], dup[s])
        tol = HALF[BF] * np.abs(D * V * slope) + 16 * U * np.abs(D * V) * (1 + gate[s].double().abs().cpu().numpy())
        near(dgate[s], torch.from_numpy(D * V * slope).cuda(), torch.from_numpy(tol).cuda(), "dgate")
    assert not bool((dgate == MARK).all(1).any()) and not bool((dup == MARK).all(1).any())


@pytest.mark.parametrize("dtype", [BF, F32])
def test_columns_of_more_workgroups_than_a_row_has(gpu_lib, dtype):
    """64 workgroups take 131072 columns of a row: those behind are a second turn's."""
    mu, g, p = gpu_lib, gen(92), 0.1
    rows, cols = 3, 131072 + 77
    x, res, y = mat(randn(g, rows, cols), dtype), mat(randn(g, rows, cols), dtype), out_mat(rows, cols, dtype)
    f = torch.from_numpy(F.dropped((rows, cols), p, *KEY)).cuda()
    mu.muon_dropout_forward(x, y, p, key_of(*KEY), residual=res)
    ref = res.double() + x.double() * f
    near(y, ref, HALF[dtype] * ref.abs() + 4 * U * (res.double().abs() + (x.double() * f).abs()), "y")
    dx, dw = out_mat(rows, cols, dtype), torch.empty((rows, 1), device="cuda")
    mu.muon_combine_backward(x, res, dx, dw, torch.ones((rows, 1), device="cuda"), p=p, key=key_of(*KEY))
    d = x.double() * f
    near(dx, d, (HALF[dtype] + 4 * U) * d.abs(), "dx")
    near(dw[:, 0], (res.double() * d).sum(1), (8 + cols / 2048 + 16) * U * (res.double() * d).abs().sum(1), "dweights")
    gate, up, dgate, dup = mat(randn(g, rows, cols), dtype), mat(randn(g, rows, cols), dtype), out_mat(rows, cols, dtype), out_mat(rows, cols, dtype)
    mu.muon_gated_backward(x, gate, up, None, None, dgate, dup)
    s = torch.sigmoid(gate.double())
    ref = x.double() * gate.double() * s
    near(dup, ref, HALF[dtype] * ref.abs() + 16 * U * (x.double() * gate.double()).abs(), "dup")
    ref = x.double() * up.double() * s * (1 + gate.double() * (1 - s))
    near(dgate, ref, HALF[dtype] * ref.abs() + 16 * U * (x.double() * up.double()).abs() * (1 + gate.double().abs()), "dgate")


def test_products_of_more_than_2_20_tiles(gpu_lib):
    """65536 groups of a slot each, 17 or more tiles across: the launch's second dimension."""
    mu, g = gpu_lib, gen(93)
    groups, n, k = 65536, 4352, 8
    w = torch.empty((groups, n, k), dtype=BF, device="cuda").normal_(0, k ** -0.5, generator=g)
    x, y = mat(randn(g, groups, k), BF), torch.full((groups, n), MARK, dtype=BF, device="cuda")
    mu.muon_expert_forward(x, w, y, torch.arange(groups + 1, dtype=torch.int32, device="cuda"))
    for lo in range(0, groups, 4096):
        terms = w[lo:lo + 4096].float() * x[lo:lo + 4096].float()[:, None, :]
        ref, mag = terms.double().sum(2), terms.double().abs().sum(2)
        near(y[lo:lo + 4096], ref, HALF[BF] * ref.abs() + (2 * k + 2) * U * mag, lo)


def test_empty_tensors_through_the_binding(gpu_lib):
    """A rank without experts, or one that no token came to: nothing is written, nothing is refused."""
    mu, g = gpu_lib, gen(94)
    i32 = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
    x, y, h = mat(randn(g, 8, 16), F32), out_mat(8, 24, F32), out_mat(8, 24, F32)
    w, none = stack(g, 2, 24, 16, F32), torch.empty((0, 24, 16), device="cuda")
    mu.muon_expert_forward(x, none, y, i32(1))
    mu.muon_gated_forward(x, none, none, h, offsets=i32(1), rows=i32(8))
    dx, grads = out_mat(8, 16, F32), [out_mat(8, 24, F32) for _ in range(2)]
    mu.muon_expert_backward(y, none, dx, i32(1))
    mu.muon_gated_backward(y, y, h, none, none, *grads, dx, i32(1), i32(8))
    ckpt = mu.Checkpoint.empty(8, 16)
    mu.muon_ckpt_save(x, ckpt)
    mu.muon_ckpt_weight_grad(y, ckpt, none, i32(1))
    # no slots: two groups of none, rows of no slots, dx of other rows
    void = [torch.empty((0, 24), device="cuda") for _ in range(5)]
    mu.muon_gated_forward(x, w, w, void[0], void[1], void[2], i32(3), i32(0), 2)
    mu.muon_gated_backward(*void[:3], w, w, *void[3:], dx, i32(3), i32(0))
    mu.muon_expert_forward(x, w, y, i32(3), i32(0), gather=1, scatter=True)
    mu.muon_expert_backward(void[0], w, dx, i32(3), i32(0), scatter=True)
    for t in (y, h, dx, *grads):
        assert bool((t == MARK).all())
    for call, a, b in ((mu.muon_expert_forward, x, y), (mu.muon_expert_backward, y, dx)):
        with pytest.raises(ValueError, match="rows: needed"):
            call(a, w, b, i32(3), gather=1, scatter=True)
