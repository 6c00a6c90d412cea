"""GPU parity of the feed-forward operators against their float64 oracles,
through the public binding, with guard rows around every matrix output.

Tolerances: half a step of the output's type relative to the value, plus a
float32 bound on the sums behind it: a sum of k products is a chain of at most
k additions, each off by u = 2^-24 of what has been added so far, which is at
most the sum of the terms' magnitudes; a matrix instruction may cut where it
adds its own products, which is twice as much; float32 products add a u each.
So (2 k + 2) u times the magnitudes. An activation's value and slope are off by
16 u of what they are made of."""
import numpy as np
import pytest
import torch

from gpu_util import padded
from oracle import ff_oracle as F

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32
HALF = {BF: 2.0 ** -8, F32: U}


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, *shape, scale=1.0):
    return torch.randn(shape, generator=g, device="cuda") * scale


def n64(t):
    return t.detach().double().cpu().numpy()


def mat(v, dtype, extra=0):
    """v in a guarded buffer of its own, rows `extra` elements longer."""
    _, t = padded(v.shape[0], v.shape[1], dtype, v.shape[1] + extra)
    t.copy_(v)
    return t


MARK = 7.0


def out_mat(rows, cols, dtype, extra=0):
    """An output full of a mark: what a call leaves alone keeps it."""
    t = padded(rows, cols, dtype, cols + extra)[1]
    t.fill_(MARK)
    return t


def stack(g, groups, rows, cols, dtype, extra=0):
    """Weights of the groups, the last guarded like the others, in one buffer with longer rows."""
    t = padded(groups * rows, cols, dtype, cols + extra)[1]
    t.copy_(randn(g, groups * rows, cols, scale=cols ** -0.5))
    return t.as_strided((groups, rows, cols), (rows * t.stride(0), t.stride(0), 1), t.storage_offset())


def close(got, ref, tol, what):
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} off, worst {np.max(np.abs(got - ref) / np.maximum(tol, 1e-300)):.3g} of the tolerance"


def lists(g, counts, topk, tokens, before=0, behind=0):
    """offsets and rows: distinct slots (token * topk + choice) in each group, ascending; slots without a group around them."""
    slots = sum(counts) + before + behind
    offsets = torch.tensor(before + np.append(0, np.cumsum(counts)), dtype=torch.int32, device="cuda")
    rows = torch.randperm(tokens * topk, generator=g, device="cuda")[:slots].to(torch.int32)
    for lo, hi in zip(offsets.tolist(), offsets.tolist()[1:]):
        rows[lo:hi] = rows[lo:hi].sort().values
    return offsets, rows


# counts of the groups' slots, n, k, longer rows: tiles of one row, of a part and of several; empty groups; widths and
# pitches of whole chunks and odd ones; sums that end inside a step and a chunk
GROUPS = [([1], 8, 8, 0), ([1, 0, 2], 1, 1, 0), ([3, 130, 0, 1, 127], 64, 32, 0), ([0, 0, 5], 136, 72, 8), ([257], 128, 40, 0),
          ([40, 60], 129, 131, 0), ([5] * 70, 24, 16, 0), ([129, 1, 300], 260, 96, 3), ([33, 0, 64], 300, 515, 0),
          ([512, 511], 256, 64, 0), ([1100], 520, 200, 0), ([2100, 5, 1500], 40, 264, 0)]


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("counts,n,k,extra", GROUPS)
def test_gated(gpu_lib, counts, n, k, extra, dtype, act):
    mu, g = gpu_lib, gen(sum(counts) + n + k)
    topk, before, behind = 3, 2, 5
    slots = sum(counts) + before + behind
    tokens = slots // topk + 2
    offsets, rows = lists(g, counts, topk, tokens, before, behind)
    rows[before::7] = -1
    x, wg, wu = mat(randn(g, tokens, k), dtype, extra), stack(g, len(counts), n, k, dtype, extra), stack(g, len(counts), n, k, dtype, extra)
    h, gate, up = (out_mat(slots, n, dtype, extra) for _ in range(3))
    mu.muon_gated_forward(x, wg, wu, h, gate, up, offsets, rows, topk, act)
    source = np.where(rows.cpu().numpy() < 0, -1, rows.cpu().numpy() // topk)
    off = offsets.tolist()
    rg, mg, used = F.product(n64(x), n64(wg), off, slots, source)
    ru, mu_, _ = F.product(n64(x), n64(wu), off, slots, source)
    eg, eu = (2 * k + 2) * U * mg, (2 * k + 2) * U * mu_
    close(n64(gate)[used], rg[used], (HALF[dtype] * np.abs(rg) + eg)[used], "gate")
    close(n64(up)[used], ru[used], (HALF[dtype] * np.abs(ru) + eu)[used], "up")
    v, _ = F.act(rg, act)
    rh = v * ru
    # slopes lie within 1.2 of 0
    th = HALF[dtype] * np.abs(rh) + 1.2 * eg * (np.abs(ru) + eu) + np.abs(v) * eu + 16 * U * np.abs(rg * ru)
    close(n64(h)[used], rh[used], th[used], "h")
    for t in (h, gate, up):
        assert np.all(n64(t)[~used] == MARK)
    alone = out_mat(slots, n, dtype)
    mu.muon_gated_forward(x, wg, wu, alone, offsets=offsets, rows=rows, rows_per_token=topk, activation=act)
    assert torch.equal(alone, h)
    # backward, from the products as stored
    dh, dgate, dup = mat(randn(g, slots, n), dtype, extra), out_mat(slots, n, dtype, extra), out_mat(slots, n, dtype, extra)
    dx = out_mat(tokens * topk, k, dtype, extra)
    mu.muon_gated_backward(dh, gate, up, wg, wu, dgate, dup, dx, offsets, rows, act)
    G, V, D = n64(gate), n64(up), n64(dh)
    v, slope = F.act(G, act)
    rdg, rdu = D * V * slope, D * v
    close(n64(dgate)[used], rdg[used], (HALF[dtype] * np.abs(rdg) + 16 * U * np.abs(D * V) * (1 + np.abs(G)))[used], "dgate")
    close(n64(dup)[used], rdu[used], (HALF[dtype] * np.abs(rdu) + 16 * U * np.abs(D * G))[used], "dup")
    assert np.all(n64(dgate)[~used] == MARK) and np.all(n64(dup)[~used] == MARK)
    a, ma, _ = F.product(n64(dgate), n64(wg), off, slots, back=True)
    b, mb, _ = F.product(n64(dup), n64(wu), off, slots, back=True)
    want, tol = np.full((tokens * topk, k), MARK), np.zeros((tokens * topk, k))
    to = rows.cpu().numpy()
    put = used & (to >= 0)
    want[to[put]] = (a + b)[put]
    tol[to[put]] = (HALF[dtype] * np.abs(a + b) + (4 * n + 2) * U * (ma + mb))[put]
    close(n64(dx), want, tol, "dx")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("slots,n,k", [(1, 300, 200), (2, 17, 33), (700, 256, 128), (1025, 384, 96), (3000, 70, 1000)])
def test_gated_dense(gpu_lib, slots, n, k, dtype):
    """One group of every row, no lists; matrices instead of stacks; no dx."""
    mu, g = gpu_lib, gen(slots + n)
    x, w = mat(randn(g, slots, k), dtype), [mat(randn(g, n, k, scale=k ** -0.5), dtype) for _ in range(2)]
    h, gate, up = (out_mat(slots, n, dtype) for _ in range(3))
    mu.muon_gated_forward(x, *w, h, gate, up)
    (rg, mg, _), (ru, mu_, _) = (F.product(n64(x), n64(m)[None], None, slots) for m in w)
    eg, eu = (2 * k + 2) * U * mg, (2 * k + 2) * U * mu_
    v, _ = F.act(rg, "silu")
    close(n64(h), v * ru, HALF[dtype] * np.abs(v * ru) + 1.2 * eg * (np.abs(ru) + eu) + np.abs(v) * eu + 16 * U * np.abs(rg * ru), "h")
    dh, dgate, dup, dx = mat(randn(g, slots, n), dtype), out_mat(slots, n, dtype), out_mat(slots, n, dtype), out_mat(slots, k, dtype)
    mu.muon_gated_backward(dh, gate, up, *w, dgate, dup, dx)
    a, ma, _ = F.product(n64(dgate), n64(w[0])[None], None, slots, back=True)
    b, mb, _ = F.product(n64(dup), n64(w[1])[None], None, slots, back=True)
    close(n64(dx), a + b, HALF[dtype] * np.abs(a + b) + (4 * n + 2) * U * (ma + mb), "dx")
    again = out_mat(slots, n, dtype), out_mat(slots, n, dtype)
    mu.muon_gated_backward(dh, gate, up, None, None, *again)
    assert torch.equal(again[0], dgate) and torch.equal(again[1], dup)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("counts,n,k,extra", GROUPS)
def test_expert(gpu_lib, counts, n, k, extra, back, dtype):
    mu, g = gpu_lib, gen(sum(counts) + n + 3 * k)
    fn = mu.muon_expert_backward if back else mu.muon_expert_forward
    topk, before, behind = 2, 1, 3
    slots = sum(counts) + before + behind
    tokens = slots // topk + 3
    offsets, rows = lists(g, counts, topk, tokens, before, behind)
    off, to = offsets.tolist(), rows.cpu().numpy()
    w = stack(g, len(counts), k if back else n, n if back else k, dtype, extra)
    x = mat(randn(g, slots, k), dtype, extra)
    r, m, used = F.product(n64(x), n64(w), off, slots, back=back)
    tol = HALF[dtype] * np.abs(r) + (2 * k + 2) * U * m
    y = out_mat(slots, n, dtype, extra)
    fn(x, w, y, offsets)
    close(n64(y)[used], r[used], tol[used], "slot order")
    assert np.all(n64(y)[~used] == MARK)
    # scattered: a row that is not named, or outside the output, is not written
    placed = out_mat(tokens * topk - 4, n, dtype, extra)
    fn(x, w, placed, offsets, rows, scatter=True)
    want, wtol = np.full(placed.shape, MARK), np.zeros(placed.shape)
    put = used & (to < len(want))
    want[to[put]], wtol[to[put]] = r[put], tol[put]
    close(n64(placed), want, wtol, "scattered")
    # gathered by token; slots of no token
    xt = mat(randn(g, tokens, k), dtype, extra)
    bad = rows.clone()
    bad[::5], bad[1::11] = -1, tokens * topk + 1
    source = np.where(bad.cpu().numpy() < 0, -1, bad.cpu().numpy() // topk)
    r, m, _ = F.product(n64(xt), n64(w), off, slots, source, back)
    y = out_mat(slots, n, dtype, extra)
    fn(xt, w, y, offsets, bad, gather=topk)
    close(n64(y)[used], r[used], (HALF[dtype] * np.abs(r) + (2 * k + 2) * U * m)[used], "gathered")
    assert np.all(n64(y)[~used] == MARK) and not n64(y)[used & ((source < 0) | (source >= tokens))].any()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_products_take_no_other_rows(gpu_lib, dtype):
    """NaN and infinities in rows of no slot, in weights of empty groups and behind a matrix's columns reach no result;
    in a slot's own row they reach that row alone."""
    mu, g = gpu_lib, gen(9)
    counts, n, k, topk = [40, 0, 25], 48, 56, 2
    slots, tokens = 65, 60
    offsets, rows = lists(g, counts, topk, tokens)
    rows[7] = rows[8]  # a token of no slot of its own is likely; make one of slot 7's rows unused
    x = mat(randn(g, tokens, k), dtype, 8)
    named = torch.zeros(tokens, dtype=torch.bool, device="cuda")
    named[(rows // topk).long()] = True
    x[~named] = float("nan")
    wg, wu = stack(g, 3, n, k, dtype, 8), stack(g, 3, n, k, dtype, 8)
    wg[1], wu[1] = float("inf"), float("nan")
    h = out_mat(slots, n, dtype)
    mu.muon_gated_forward(x, wg, wu, h, offsets=offsets, rows=rows, rows_per_token=topk)
    assert bool(torch.isfinite(h).all())
    x[int(rows[30]) // topk, 3] = float("inf")
    h2 = out_mat(slots, n, dtype)
    mu.muon_gated_forward(x, wg, wu, h2, offsets=offsets, rows=rows, rows_per_token=topk)
    hit = (rows // topk) == rows[30] // topk
    assert torch.equal(h2[~hit], h[~hit]) and not bool(torch.isfinite(h2[hit]).any())


@pytest.mark.parametrize("dtype", [BF, F32])
def test_products_of_nothing(gpu_lib, dtype):
    """No slots, no groups, no tokens; offsets outside the slots; sums with no row of x."""
    mu, g = gpu_lib, gen(11)
    w = stack(g, 2, 16, 24, dtype)
    none = torch.tensor([0, 0, 0], dtype=torch.int32, device="cuda")
    x, y = mat(randn(g, 30, 24), dtype), out_mat(30, 16, dtype)
    mu.muon_expert_forward(x, w, y, none)
    assert bool((y == MARK).all())
    mu.muon_expert_forward(x[:0], w, y[:0], none)
    mu.muon_gated_forward(x[:0], w, w.clone(), y[:0], offsets=none)
    wild = torch.tensor([-5, 11, 99], dtype=torch.int32, device="cuda")
    mu.muon_expert_forward(x, w, y, wild)
    plain = torch.tensor([0, 11, 30], dtype=torch.int32, device="cuda")
    z = out_mat(30, 16, dtype)
    mu.muon_expert_forward(x, w, z, plain)
    assert torch.equal(y, z)
    rows = torch.arange(30, dtype=torch.int32, device="cuda")
    mu.muon_gated_forward(x[:0], w, w.clone(), z, offsets=plain, rows=rows)
    mu.muon_expert_forward(x[:0], w, y, plain, rows, gather=1)
    assert not bool(z.any()) and not bool(y.any())


KEY = (0x1234567890ABCDEF, 0x0FEDCBA987654321)


def key_of(seed, offset):
    return torch.tensor([seed, offset], dtype=torch.int64, device="cuda")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("p", [0.0, 0.1, 0.9999])
@pytest.mark.parametrize("rows,cols,extra", [(1, 1, 0), (3, 5, 2), (300, 1, 0), (17, 64, 0), (33, 65, 0), (9, 512, 8),
                                             (5, 2047, 0), (4, 2053, 3), (2, 70001, 0), (1000, 7, 0)])
def test_dropout(gpu_lib, rows, cols, extra, p, dtype):
    mu, g = gpu_lib, gen(rows + cols)
    x, res, y = mat(randn(g, rows, cols), dtype, extra), mat(randn(g, rows, cols), dtype, extra), out_mat(rows, cols, dtype, extra)
    key = key_of(*KEY)
    f = F.dropped((rows, cols), p, *KEY)
    mu.muon_dropout_forward(x, y, p, key if p else None, residual=res)
    ref = n64(res) + n64(x) * f
    # a product with the rounded 1 / (1 - p), and a sum
    close(n64(y), ref, HALF[dtype] * np.abs(ref) + 4 * U * (np.abs(n64(res)) + np.abs(n64(x) * f)), "y")
    for call, out in ((mu.muon_dropout_forward, out_mat(rows, cols, dtype)), (mu.muon_dropout_backward, out_mat(rows, cols, dtype))):
        call(x, out, p, key)
        close(n64(out), n64(x) * f, (HALF[dtype] + 4 * U) * np.abs(n64(x) * f), call.__name__)
        assert np.array_equal(n64(out) == 0, (f == 0) | (n64(x) == 0))


def test_dropout_words_against_published_ones(gpu_lib):
    """Which elements stay, at a threshold that falls between known words of Philox4x32-10 (the authors' test vectors:
    zeros, ones, digits of pi)."""
    for counter, key, words in (
            ((0, 0, 0, 0), (0, 0), (0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8)),
            ((0xffffffff,) * 4, (0xffffffff,) * 2, (0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd)),
            ((0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344), (0xa4093822, 0x299f31d0), (0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1))):
        assert tuple(int(v) for v in F.philox(counter, key)) == words
    x, y = torch.ones((1, 4), device="cuda"), torch.empty((1, 4), device="cuda")
    for p in np.linspace(0.01, 0.99, 23):
        gpu_lib.muon_dropout_forward(x, y, float(p), key_of(0, 0))
        words = np.array([0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8])
        assert np.array_equal(n64(y)[0] != 0, words >= float(np.float32(p)) * 2 ** 32)


def test_dropout_far_into_the_counter(gpu_lib):
    """Elements past 2^32, and rows whose buffer passes 2^31 elements."""
    mu = gpu_lib
    rows, cols = 70001, 65537
    assert rows * cols > 2 ** 32
    x = torch.ones((rows, cols), dtype=BF, device="cuda")
    y = torch.empty_like(x)
    mu.muon_dropout_forward(x, y, 0.5, key_of(*KEY))
    for r in (0, 1, 32768, 65535, 65536, 70000):
        want = F.kept(r * cols, cols, 0.5, *KEY)
        assert np.array_equal(y[r].float().cpu().numpy() != 0, want), r
    share = float((y[::1000] != 0).float().mean())
    assert abs(share - 0.5) < 1e-3  # 4.6 million fair draws: 4 sigma


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("tokens,topk,cols,extra,p", [(1, 1, 1, 0, 0.3), (5, 3, 7, 0, 0.0), (100, 8, 64, 0, 0.1), (33, 9, 65, 3, 0.5),
                                                      (40, 2, 511, 0, 0.1), (7, 32, 600, 8, 0.2), (21, 8, 2048, 0, 0.1),
                                                      (3, 17, 4101, 0, 0.1), (600, 4, 16, 0, 0.25)])
def test_combine(gpu_lib, tokens, topk, cols, extra, p, weighted, dtype):
    mu, g = gpu_lib, gen(tokens + topk + cols)
    slots = tokens * topk
    x, res = mat(randn(g, slots, cols), dtype, extra), mat(randn(g, tokens, cols), dtype, extra)
    y, key = out_mat(tokens, cols, dtype, extra), key_of(*KEY)
    w = torch.rand((tokens, topk), generator=g, device="cuda") if weighted else None
    idx = torch.randint(0, 9, (tokens, topk), generator=g, device="cuda").to(torch.int32)
    idx[torch.rand(idx.shape, generator=g, device="cuda") < 0.2] = -1
    idx[tokens // 2] = -1  # a token without any choice
    there = idx.cpu().numpy() >= 0
    x[torch.from_numpy(~there.reshape(-1)).cuda()] = float("nan")  # rows that do not count
    mu.muon_combine_forward(x, y, w, idx, res, p, key)
    W = (n64(w) if weighted else np.ones((tokens, topk))) * there
    X = np.where(there[:, :, None], n64(x).reshape(tokens, topk, cols), 0.0)
    f = F.dropped((tokens, cols), p, *KEY)
    total, mag = (W[:, :, None] * X).sum(1), np.abs(W[:, :, None] * X).sum(1)
    ref = n64(res) + total * f
    close(n64(y), ref, HALF[dtype] * np.abs(ref) + U * (np.abs(n64(res)) + (topk + 4) * mag * f), "y")
    # backward: in x's order, then in the order of a list that leaves out what does not count
    dy, dx, dw = mat(randn(g, tokens, cols), dtype, extra), out_mat(slots, cols, dtype, extra), torch.full((tokens, topk), MARK, device="cuda")
    mu.muon_combine_backward(dy, x, dx, dw if weighted else None, w, idx, None, p, key)
    d = n64(dy) * f
    rdx = (W[:, :, None] * d[:, None]).reshape(slots, cols)
    live = there.reshape(-1)
    close(n64(dx)[live], rdx[live], (HALF[dtype] + 4 * U) * np.abs(rdx)[live], "dx")
    assert np.all(n64(dx)[~live] == MARK)
    if weighted:
        # eight products in turn a run, the runs of a thread, sums over 256 threads
        rdw, mag = (X * d[:, None]).sum(2), np.abs(X * d[:, None]).sum(2)
        close(n64(dw), rdw, (8 + cols / 2048 + 16) * U * mag, "dweights")
        assert not n64(dw)[~there].any()
    perm = torch.from_numpy(np.random.RandomState(tokens).permutation(np.flatnonzero(live))).to(torch.int32).cuda()
    rows = torch.cat([perm, torch.full((slots - len(perm),), -1, dtype=torch.int32, device="cuda")])
    listed, dw2 = out_mat(slots, cols, dtype, extra), torch.full((tokens, topk), MARK, device="cuda")
    mu.muon_combine_backward(dy, x, listed, dw2 if weighted else None, w, idx, rows, p, key)
    assert torch.equal(listed[:len(perm)], dx[perm.long()]) and bool((listed[len(perm):] == MARK).all())
    assert not weighted or torch.equal(dw, dw2)


def test_combine_of_a_partial_list(gpu_lib):
    """Slots that the list does not name write no row, whatever the workspace holds; entries outside the slots count as none."""
    mu, g = gpu_lib, gen(21)
    tokens, topk, cols = 50, 4, 96
    dy, slots = mat(randn(g, tokens, cols), F32), tokens * topk
    rows = torch.full((slots,), -1, dtype=torch.int32, device="cuda")
    rows[10:60] = torch.randperm(slots, generator=g, device="cuda")[:50].to(torch.int32)
    rows[70], rows[71] = slots, 2 ** 31 - 1
    for fill in (0, 12, 255):
        ws = torch.full((mu.muon_combine_workspace_size(tokens, topk),), fill, dtype=torch.uint8, device="cuda")
        dx = out_mat(slots, cols, F32)
        mu.muon_combine_backward(dy, None, dx, rows=rows, workspace=ws)
        assert torch.equal(dx[10:60], dy[(rows[10:60] // topk).long()])
        assert bool((dx[:10] == MARK).all()) and bool((dx[60:] == MARK).all())


def test_dropped_values_do_not_count(gpu_lib):
    """NaN and infinities in dropped places leave zeros, forward and backward."""
    mu, g = gpu_lib, gen(22)
    rows, cols, p = 40, 300, 0.4
    f = torch.from_numpy(F.dropped((rows, cols), p, *KEY)).cuda()
    x = mat(randn(g, rows, cols), F32)
    x[f == 0] = float("nan")
    key, y, dx = key_of(*KEY), out_mat(rows, cols, F32), out_mat(rows, cols, F32)
    mu.muon_dropout_forward(x, y, p, key)
    mu.muon_dropout_backward(x, dx, p, key)
    assert bool((y[f == 0] == 0).all()) and bool(torch.isfinite(y).all()) and torch.equal(y, dx)
    dw = torch.empty((rows, 1), device="cuda")
    good = mat(randn(g, rows, cols), F32)
    mu.muon_combine_backward(good, x, dx, dw, weights=torch.ones((rows, 1), device="cuda"), p=p, key=key)
    assert bool(torch.isfinite(dw).all())


# ---------------------------------------------------------------------------
# sizes that take every form of tile, against 64-bit products on the GPU
# ---------------------------------------------------------------------------

def grouped64(x, w, offsets, source, back):
    """(products, magnitudes) in slot order, in 64 bits on the GPU."""
    cols = w.shape[2] if back else w.shape[1]
    y = torch.zeros((len(source), cols), dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(y)
    for g, (lo, hi) in enumerate(zip(offsets, offsets[1:])):
        if hi > lo:
            m = w[g].double() if back else w[g].double().t().contiguous()
            rows = x[source[lo:hi].clamp(min=0)].double() * (source[lo:hi] >= 0)[:, None]
            y[lo:hi], mag[lo:hi] = rows @ m, rows.abs() @ m.abs()
    return y, mag


def near(got, ref, tol, what):
    bad = ~((got.double() - ref).abs() <= tol)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} off, worst {float(((got.double() - ref).abs() / tol.clamp(min=1e-300)).max()):.3g} of the tolerance"


# tokens, topk, experts, n, k: tiles of every size, two row halves, one group and many; the same with rows that start on no
# 16-byte boundary. Of 256 x 256 tiles that stream there is the gated forward pass of 5000 tokens; the other kinds' are in
# test_gpu_ff_forms.py.
SIZES = [(9000, 1, 1, 2304, 128), (5000, 4, 40, 640, 192), (4000, 2, 600, 264, 64), (900, 8, 128, 256, 64), (2300, 1, 1, 2048, 64),
         (700, 1, 1, 1024, 256), (513, 3, 16, 200, 512), (60, 4, 64, 512, 320), (2, 1, 1, 4096, 1024), (9, 2, 35, 72, 2048),
         (8000, 1, 1, 2303, 127), (5000, 4, 40, 639, 191), (2300, 1, 1, 2047, 63), (1000, 2, 30, 201, 333), (3, 2, 9, 515, 1031)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("tokens,topk,experts,n,k", SIZES)
def test_products_of_every_size(gpu_lib, tokens, topk, experts, n, k, dtype):
    mu, g = gpu_lib, gen(tokens + experts + n)
    slots = tokens * topk
    # uneven groups, some of them empty, some slots behind the last
    share = torch.rand(experts, generator=g, device="cuda") ** 2 * (torch.rand(experts, generator=g, device="cuda") < 0.9)
    ends = (share.cumsum(0) / share.sum().clamp(min=1e-3) * (slots - slots // 50)).long() if experts > 1 else torch.tensor([slots], device="cuda")
    offsets = torch.cat([ends.new_zeros(1), ends]).to(torch.int32)
    rows = torch.randperm(slots, generator=g, device="cuda").to(torch.int32)
    rows[::97] = -1
    off = offsets.tolist()
    used = torch.arange(slots, device="cuda") < off[-1]
    token = torch.where(rows < 0, -1, rows // topk).long()
    x, wg, wu = mat(randn(g, tokens, k), dtype), stack(g, experts, n, k, dtype), stack(g, experts, n, k, dtype)
    h, gate, up = (out_mat(slots, n, dtype) for _ in range(3))
    mu.muon_gated_forward(x, wg, wu, h, gate, up, offsets, rows, topk)
    rg, mg = grouped64(x, wg, off, token, False)
    ru, mu_ = grouped64(x, wu, off, token, False)
    u = (2 * k + 2) * U
    near(gate[used], rg[used], (HALF[dtype] * rg.abs() + u * mg)[used], "gate")
    near(up[used], ru[used], (HALF[dtype] * ru.abs() + u * mu_)[used], "up")
    v = rg * torch.sigmoid(rg)
    near(h[used], (v * ru)[used], (HALF[dtype] * (v * ru).abs() + 1.2 * u * mg * (ru.abs() + u * mu_) + v.abs() * u * mu_ +
                                   16 * U * (rg * ru).abs())[used], "h")
    assert bool((h[~used] == MARK).all() and (gate[~used] == MARK).all() and (up[~used] == MARK).all())
    del rg, mg, ru, mu_, v
    dh, dgate, dup = mat(randn(g, slots, n), dtype), out_mat(slots, n, dtype), out_mat(slots, n, dtype)
    dx = out_mat(slots, k, dtype)
    mu.muon_gated_backward(dh, gate, up, wg, wu, dgate, dup, dx, offsets, rows)
    own = torch.arange(slots, device="cuda")
    a, ma = grouped64(dgate, wg, off, own, True)
    b, mb = grouped64(dup, wu, off, own, True)
    put = used & (rows >= 0)
    near(dx[rows[put].long()], (a + b)[put], (HALF[dtype] * (a + b).abs() + (4 * n + 2) * U * (ma + mb))[put], "dx")
    other = torch.ones(slots, dtype=torch.bool, device="cuda")
    other[rows[put].long()] = False
    assert bool((dx[other] == MARK).all())
    del a, b, ma, mb
    for back in (False, True):
        xs = mat(randn(g, slots, n if back else k), dtype)
        y = out_mat(slots, k if back else n, dtype)
        (mu.muon_expert_backward if back else mu.muon_expert_forward)(xs, wg, y, offsets)
        r, m = grouped64(xs, wg, off, own, back)
        near(y[used], r[used], (HALF[dtype] * r.abs() + (2 * xs.shape[1] + 2) * U * m)[used], "backward" if back else "forward")
        assert bool((y[~used] == MARK).all())


# Its 70000 rows take 128 x 256 tiles by the plan as it is; tiles that stream whose sums end inside a step: test_gpu_ff_forms.py.
@pytest.mark.parametrize("k", [33, 40, 63, 64, 65, 72, 96, 120, 129, 200])
def test_products_whose_sum_ends_anywhere_in_a_step(gpu_lib, k):
    """The operands lie in buffers of NaN: nothing behind a sum's end takes part. Tiles that stream (enough rows for them),
    small ones and those of registers."""
    mu, g = gpu_lib, gen(k)
    for rows, n in ((70000, 264), (130, 264), (20, 24)):
        for dtype in (BF, F32):
            wide = torch.full((rows + 2, 256), float("nan"), dtype=dtype, device="cuda")
            x = wide[1:-1, :k]
            x.copy_(randn(g, rows, k))
            wbuf = torch.full((n + 2, 256), float("nan"), dtype=dtype, device="cuda")
            w = wbuf[1:-1, :k]
            w.copy_(randn(g, n, k, scale=k ** -0.5))
            y = out_mat(rows, n, dtype)
            mu.muon_expert_forward(x, w, y)
            r, m = grouped64(x, w[None], [0, rows], torch.arange(rows, device="cuda"), False)
            near(y, r, HALF[dtype] * r.abs() + (2 * k + 2) * U * m, f"forward {rows} {dtype}")
            # backward: the sum's index is the weights' row
            wt = torch.full((k + 2, 320), float("nan"), dtype=dtype, device="cuda")
            v = wt[1:-1, :n]
            v.copy_(w.t())
            z = out_mat(rows, n, dtype)
            mu.muon_expert_backward(x, v, z)
            near(z, r, HALF[dtype] * r.abs() + (2 * k + 2) * U * m, f"backward {rows} {dtype}")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("tokens,n,k", [(40, 24, 40), (700, 130, 65), (21, 16, 8200)])
def test_lists_without_groups(gpu_lib, tokens, n, k, dtype):
    """One matrix of weights, no offsets: rows alone gather, scatter and do both; a longer list of a token's entries than one."""
    mu, g, topk = gpu_lib, gen(tokens + k), 2
    slots = tokens * topk
    rows = torch.randperm(slots, generator=g, device="cuda").to(torch.int32)
    rows[3::17] = -1
    there = rows >= 0
    x, w = mat(randn(g, tokens, k), dtype), mat(randn(g, n, k, scale=k ** -0.5), dtype)
    r, m = grouped64(x, w[None], [0, slots], torch.where(there, rows // topk, -1).long(), False)
    tol = HALF[dtype] * r.abs() + (2 * k + 2) * U * m
    y = out_mat(slots, n, dtype)
    mu.muon_expert_forward(x, w, y, rows=rows, gather=topk)
    near(y, r, tol, "gathered")
    z = out_mat(slots, n, dtype)
    mu.muon_expert_forward(x, w, z, rows=rows, gather=topk, scatter=True)
    assert torch.equal(z[rows[there].long()], y[there])
    other = torch.ones(slots, dtype=torch.bool, device="cuda")
    other[rows[there].long()] = False
    assert bool((z[other] == MARK).all())
    h, one = out_mat(slots, n, dtype), mat(randn(g, n, k, scale=k ** -0.5), dtype)
    mu.muon_gated_forward(x, w, one, h, rows=rows, rows_per_token=topk)
    u, mu_ = grouped64(x, one[None], [0, slots], torch.where(there, rows // topk, -1).long(), False)
    v, e, eu = r * torch.sigmoid(r), (2 * k + 2) * U * m, (2 * k + 2) * U * mu_
    near(h, v * u, HALF[dtype] * (v * u).abs() + 1.2 * e * (u.abs() + eu) + v.abs() * eu + 16 * U * (r * u).abs(), "gated")


# tokens, topk, experts, width, length of the sum: few outputs of long sums, which several workgroups share. The bounds below
# are the worst case of each value; test_gpu_ff_forms.py holds the same sizes to float32 sums in norm.
LONG = [(1, 1, 1, 5, 8192), (64, 1, 1, 520, 8192), (100, 3, 4, 129, 4095), (40, 1, 3, 72, 6001), (33, 2, 9, 64, 12288),
        (12, 2, 5, 72, 8001), (16, 2, 3, 264, 9000)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("tokens,topk,experts,n,k", LONG)
def test_long_sums_shared_out(gpu_lib, tokens, topk, experts, n, k, dtype):
    """The parts go to a workspace of exactly the size asked for, full of NaN; slots of no group or token; an infinity in one
    slot; the same bits twice; too little workspace is refused."""
    mu, g = gpu_lib, gen(tokens + n + k)
    code = mu.MUON_BF16 if dtype == BF else mu.MUON_F32
    slots = tokens * topk
    ends = torch.arange(experts + 1, device="cuda") * (slots - (2 if experts > 1 else 0)) // experts
    ends[0] = 1 if experts > 1 else 0
    offsets, off = ends.to(torch.int32), ends.tolist()
    rows = torch.randperm(slots, generator=g, device="cuda").to(torch.int32)
    if experts > 1:
        rows[5::11] = -1
    token = torch.where(rows < 0, -1, rows // topk).long()
    own = torch.arange(slots, device="cuda")
    used = (own >= off[0]) & (own < off[-1])

    def twice(size, fn, *outs):
        assert size > 0
        buf = torch.full((size + 4096,), 255, dtype=torch.uint8, device="cuda")
        ws = buf[:size]
        fn(ws)
        first = [o.clone() for o in outs]
        ws.fill_(255)
        fn(ws)
        for a, b in zip(first, outs):
            assert torch.equal(a.nan_to_num(), b.nan_to_num())
        with pytest.raises(mu.MuonError, match="workspace"):
            fn(ws[:size - 4])
        assert bool((buf[size:] == 255).all())

    # forward, gated: sums of k
    x, wg, wu = mat(randn(g, tokens, k), dtype), stack(g, experts, n, k, dtype), stack(g, experts, n, k, dtype)
    h, gate, up = (out_mat(slots, n, dtype) for _ in range(3))
    twice(mu.muon_gated_workspace_size(code, slots, n, k, experts), lambda ws: mu.muon_gated_forward(
        x, wg, wu, h, gate, up, offsets, rows, topk, workspace=ws), h, gate, up)
    rg, mg = grouped64(x, wg, off, token, False)
    ru, mu_ = grouped64(x, wu, off, token, False)
    u = (2 * k + 2) * U
    near(gate[used], rg[used], (HALF[dtype] * rg.abs() + u * mg)[used], "gate")
    near(up[used], ru[used], (HALF[dtype] * ru.abs() + u * mu_)[used], "up")
    v = rg * torch.sigmoid(rg)
    near(h[used], (v * ru)[used], (HALF[dtype] * (v * ru).abs() + 1.2 * u * mg * (ru.abs() + u * mu_) + v.abs() * u * mu_ +
                                   16 * U * (rg * ru).abs())[used], "h")
    assert bool((h[~used] == MARK).all() and (gate[~used] == MARK).all() and (up[~used] == MARK).all())
    only = out_mat(slots, n, dtype)
    mu.muon_gated_forward(x, wg, wu, only, offsets=offsets, rows=rows, rows_per_token=topk)  # a workspace of the binding's
    assert torch.equal(only, h)
    # forward, scattered; an infinity stays in its slot
    xs, y = mat(randn(g, slots, k), dtype), out_mat(slots, n, dtype)
    at = off[0] + (off[-1] - off[0]) // 2
    xs[at, 7] = float("inf")
    twice(mu.muon_expert_workspace_size(code, slots, n, k, experts), lambda ws: mu.muon_expert_forward(
        xs, wg, y, offsets, rows, scatter=True, workspace=ws), y)
    r, m = grouped64(xs, wg, off, own, False)
    put = used & (rows >= 0)
    to = rows[put].long()
    if int(rows[at]) >= 0:
        assert not bool(torch.isfinite(y[int(rows[at])]).any())
    put[at] = False
    near(y[rows[put].long()], r[put], (HALF[dtype] * r.abs() + u * m)[put], "scattered")
    other = torch.ones(slots, dtype=torch.bool, device="cuda")
    other[to] = False
    assert bool((y[other] == MARK).all())
    # backward: the weights' rows are summed over
    wd, we = stack(g, experts, k, n, dtype), stack(g, experts, k, n, dtype)
    xs = mat(randn(g, slots, k), dtype)
    y = out_mat(slots, n, dtype)
    twice(mu.muon_expert_workspace_size(code, slots, k, n, experts, 1), lambda ws: mu.muon_expert_backward(
        xs, wd, y, offsets, workspace=ws), y)
    r, m = grouped64(xs, wd, off, own, True)
    near(y[used], r[used], (HALF[dtype] * r.abs() + u * m)[used], "backward")
    assert bool((y[~used] == MARK).all())
    # both products' gradient of x, one sum
    gate, up, dh = (mat(randn(g, slots, k), dtype) for _ in range(3))
    dgate, dup, dx = out_mat(slots, k, dtype), out_mat(slots, k, dtype), out_mat(slots, n, dtype)
    twice(mu.muon_gated_workspace_size(code, slots, k, n, experts, 1), lambda ws: mu.muon_gated_backward(
        dh, gate, up, wd, we, dgate, dup, dx, offsets, rows, workspace=ws), dx)
    a, ma = grouped64(dgate, wd, off, own, True)
    b, mb = grouped64(dup, we, off, own, True)
    put = used & (rows >= 0)
    near(dx[rows[put].long()], (a + b)[put], (HALF[dtype] * (a + b).abs() + (4 * k + 2) * U * (ma + mb))[put], "dx")
    assert bool((dx[other] == MARK).all())


# tokens, width, length of the sum: one group's tiles that go round the CUs once and a little more. Swapped for the backward
# products. The last with rows that start on no 16-byte boundary.
LEFT_OVER = [(33, 17000, 640, F32), (500, 2060, 1024, F32), (33, 17000, 3686, BF), (33, 17000, 7168, BF),
             (33, 17003, 643, F32), (33, 17005, 3689, BF)]


@pytest.mark.parametrize("swapped", [False, True])
@pytest.mark.parametrize("tokens,n,k,dtype", LEFT_OVER)
def test_columns_left_over_are_shared_out(gpu_lib, tokens, n, k, dtype, swapped):
    mu, code = gpu_lib, gpu_lib.MUON_BF16 if dtype == BF else gpu_lib.MUON_F32
    w = (k, n) if swapped else (n, k)
    sizes = [f(code, tokens, *w, 1, int(swapped)) / (tokens * n * 4) for f in (mu.muon_gated_workspace_size, mu.muon_expert_workspace_size)]
    assert any(size % 1 for size in sizes), sizes  # parts of some of the columns
    test_products_of_every_size(mu, tokens, 1, 1, *w, dtype)


def test_long_sums_captured(gpu_lib):
    """Two graphs whose parts lie in one workspace, replayed in turn on new inputs, as eager calls."""
    mu, g, n, k = gpu_lib, gen(3), 72, 8192
    ws = torch.empty(mu.muon_gated_workspace_size(mu.MUON_F32, 40, n, k), dtype=torch.uint8, device="cuda")
    sets = []
    for i in range(2):
        x, wg, wu, h = mat(randn(g, 40, k), F32), stack(g, 1, n, k, F32)[0], stack(g, 1, n, k, F32)[0], out_mat(40, n, F32)
        mu.muon_gated_forward(x, wg, wu, h, workspace=ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            mu.muon_gated_forward(x, wg, wu, h, workspace=ws)
        sets.append((graph, x, wg, wu, h))
    for _ in range(3):
        for graph, x, wg, wu, h in sets:
            x.copy_(randn(g, 40, k))
            h.fill_(MARK)
            graph.replay()
            want = out_mat(40, n, F32)
            mu.muon_set_stream(torch.cuda.current_stream().cuda_stream)
            mu.muon_gated_forward(x, wg, wu, want)
            torch.cuda.synchronize()
            assert torch.equal(h, want)
    mu.muon_set_stream(None)
