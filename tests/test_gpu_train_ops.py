"""GPU parity of the training operators against their float64 oracles, through
the public binding, with guard rows around every matrix output.

Tolerances: half a step of the output's type relative to the value, plus a
float32 bound on the sums behind it: u = 2^-24 times the length of the longest
chain of additions (and the few roundings of each term) times the sum of the
terms' magnitudes. Codes, scales, indices, counts and lists are exact."""
import numpy as np
import pytest
import torch

from gpu_util import padded
from oracle import train_oracle as T

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


def out_mat(rows, cols, dtype, extra=0):
    return padded(rows, cols, dtype, cols + extra)[1]


class Codes:
    """A checkpoint whose codes and scales lie inside larger buffers of a known fill."""

    def __init__(self, mu, rows, cols, extra=0):
        groups = -(-cols // 128)
        self.c = torch.full((rows + 2, cols + extra), 0x55, dtype=torch.uint8, device="cuda")
        self.s = torch.full((rows + 2, groups + extra), 0x55, dtype=torch.uint8, device="cuda")
        self.rows, self.cols, self.groups = rows, cols, groups
        self.ck = mu.Checkpoint(self.c.view(torch.float8_e4m3fn)[1:1 + rows, :cols], self.s[1:1 + rows, :groups])

    def check(self):
        for t, cols in ((self.c, self.cols), (self.s, self.groups)):
            assert bool((t[0] == 0x55).all() and (t[self.rows + 1:] == 0x55).all() and (t[:, cols:] == 0x55).all())

    def read(self):
        v = T.code_values()[self.c[1:1 + self.rows, :self.cols].cpu().numpy()]
        return v, self.s[1:1 + self.rows, :self.groups].cpu().numpy().astype(np.int64)


def close(got, ref, tol, what):
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} off, worst {np.max(np.abs(got - ref) / np.maximum(tol, 1e-300)):.3g} of the tolerance"


# rows, cols, pitch beyond cols: each width class of the kernels, odd widths and pitches, one row and one column
NORM = [(1, 1, 0), (3, 7, 0), (5, 129, 3), (37, 512, 0), (9, 513, 0), (64, 1024, 8), (13, 1025, 1), (4, 2048, 0),
        (33, 2047, 0), (21, 4096, 0), (7, 4097, 5), (130, 7168, 0), (3, 8193, 0), (2, 16385, 1), (2, 32768, 0)]


@pytest.mark.parametrize("dtype,wdtype", [(BF, BF), (BF, F32), (F32, F32), (F32, BF)])
@pytest.mark.parametrize("rows,cols,extra", NORM)
def test_layernorm(gpu_lib, rows, cols, extra, dtype, wdtype):
    mu, g = gpu_lib, gen(rows * 40000 + cols)
    x = mat(randn(g, rows, cols) * 2 + 0.7, dtype, extra)
    w, b = mat(1 + randn(g, 1, cols, scale=0.3), wdtype), mat(randn(g, 1, cols, scale=0.3), wdtype)
    dy = mat(randn(g, rows, cols, scale=1e-2), dtype, extra)
    y, dx = out_mat(rows, cols, dtype, extra), out_mat(rows, cols, dtype, extra)
    dw, db = out_mat(1, cols, wdtype), out_mat(1, cols, wdtype)
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    codes = Codes(mu, rows, cols, extra)
    mu.muon_layernorm_forward(x, y, mean, rstd, w, b, eps=1e-5, ckpt=codes.ck)
    X, W, B = n64(x), n64(w)[0], n64(b)[0]
    ry, rm, rr = T.layernorm(X, W, B)
    big = np.abs(X).max(1)
    # the mean: tree sums of at most 32 terms a thread, then 6 + 4 levels
    close(n64(mean), rm, 48 * U * np.abs(X).mean(1), "mean")
    close(n64(rstd), rr, 48 * U * rr * (1 + rr * big), "rstd")
    scale = ((big + np.abs(rm)) * rr)[:, None] * np.abs(W)
    close(n64(y), ry, HALF[dtype] * np.abs(ry) + 48 * U * (scale * (1 + (rr * big)[:, None]) + np.abs(B)), "y")
    # the checkpoint of y as stored, bit for bit
    unit, sb = T.checkpoint(n64(y))
    got, gb = codes.read()
    codes.check()
    assert np.array_equal(gb, sb) and np.array_equal(got, unit)
    # backward, from the statistics as stored
    mu.muon_layernorm_backward(dy, x, mean, rstd, dx, w, dw, db)
    D, M, R = n64(dy), n64(mean), n64(rstd)
    rdx, rdw, rdb = T.layernorm_grad(D, X, M, R, W)
    xh, h = (X - M[:, None]) * R[:, None], D * W
    mag = R[:, None] * (np.abs(h) + np.abs(h).mean(1, keepdims=True) + np.abs(xh) * np.abs(h * xh).mean(1, keepdims=True))
    slack = (1 + (R * big)[:, None])  # x - mean is rounded against x
    close(n64(dx), rdx, HALF[dtype] * np.abs(rdx) + 64 * U * mag * slack, "dx")
    # at most 32 rows a chain here, 4 waves, 64 partials in 8 slices
    close(n64(dw)[0], rdw, HALF[wdtype] * np.abs(rdw) + 128 * U * (np.abs(D * xh) * slack).sum(0), "dweight")
    close(n64(db)[0], rdb, HALF[wdtype] * np.abs(rdb) + 128 * U * np.abs(D).sum(0), "dbias")


def test_layernorm_many_rows_and_optional_operands(gpu_lib):
    """More rows than workgroups; no weight, no bias, no statistics, one gradient alone; no rows at all."""
    mu, g = gpu_lib, gen(5)
    rows, cols = 9001, 96
    x, dy = mat(randn(g, rows, cols), BF), mat(randn(g, rows, cols), BF)
    y, dx = out_mat(rows, cols, BF), out_mat(rows, cols, BF)
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    mu.muon_layernorm_forward(x, y, mean, rstd)
    y2 = out_mat(rows, cols, BF)
    mu.muon_layernorm_forward(x, y2)
    assert torch.equal(y, y2)
    ry, _, _ = T.layernorm(n64(x))
    close(n64(y), ry, 2.0 ** -8 * np.abs(ry) + 64 * U * (1 + np.abs(ry)) ** 2, "y")
    db, dw = out_mat(1, cols, F32), out_mat(1, cols, F32)
    mu.muon_layernorm_backward(dy, x, mean, rstd, dx, dbias=db)
    mu.muon_layernorm_backward(dy, x, mean, rstd, dx, dweight=dw)
    M, R = n64(mean), n64(rstd)
    _, rdw, rdb = T.layernorm_grad(n64(dy), n64(x), M, R)
    xh = (n64(x) - M[:, None]) * R[:, None]
    close(n64(db)[0], rdb, 128 * U * np.abs(n64(dy)).sum(0), "dbias")
    close(n64(dw)[0], rdw, 128 * U * (np.abs(n64(dy) * xh) + np.abs(n64(dy))).sum(0), "dweight")
    only = out_mat(rows, cols, BF)
    mu.muon_layernorm_backward(dy, x, mean, rstd, only)
    assert torch.equal(only, dx)
    none = torch.empty((0, cols), dtype=BF, device="cuda")
    stat = torch.empty(0, device="cuda")
    mu.muon_layernorm_forward(none, none.clone(), stat, stat.clone())
    mu.muon_layernorm_backward(none, none.clone(), stat, stat.clone(), none.clone(), dweight=dw, dbias=db)
    assert not n64(dw).any() and not n64(db).any()


def test_layernorm_infinities_stay_in_their_row(gpu_lib):
    x = mat(randn(gen(6), 4, 300), F32)
    x[1, 7], x[2, 3] = float("inf"), float("nan")
    y = out_mat(4, 300, F32, 0)
    codes = Codes(gpu_lib, 4, 300)
    gpu_lib.muon_layernorm_forward(x, y, ckpt=codes.ck)
    assert bool(torch.isnan(y[1]).all() and torch.isnan(y[2]).all() and torch.isfinite(y[0]).all() and torch.isfinite(y[3]).all())
    got, _ = codes.read()
    assert np.isnan(got[1]).all() and np.isfinite(got[0]).all()


CKPT = [(1, 1, 0), (2, 5, 0), (3, 128, 0), (5, 129, 1), (17, 255, 7), (100, 768, 0), (31, 2047, 0), (9, 7168, 0), (300, 40, 0)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,cols,extra", CKPT)
def test_checkpoint(gpu_lib, rows, cols, extra, dtype):
    mu, g = gpu_lib, gen(rows * 40000 + cols)
    v = randn(g, rows, cols) * torch.exp(2 * randn(g, 1, cols))
    v[torch.rand(v.shape, generator=g, device="cuda") < 0.02] = 0
    x = mat(v, dtype, extra)
    codes = Codes(mu, rows, cols, extra)
    mu.muon_ckpt_save(x, codes.ck)
    unit, sb = T.checkpoint(n64(x))
    got, gb = codes.read()
    codes.check()
    assert np.array_equal(gb, sb) and np.array_equal(got, unit)
    for to in (BF, F32):
        back = out_mat(rows, cols, to, extra)
        mu.muon_ckpt_load(codes.ck, back)
        assert np.array_equal(n64(back), T.values(unit, sb)), to


def test_checkpoint_of_special_values(gpu_lib):
    """Zeros, denormals, the largest values, infinities and NaN, ties and both sides of a scale's border."""
    rows = torch.zeros((8, 256), device="cuda")
    rows[1, :4] = torch.tensor([float("inf"), 1.0, -float("inf"), float("nan")], device="cuda")
    rows[2, 0], rows[2, 128] = 3.4028234e38, 1e-45
    rows[3, 0], rows[3, 128] = 1.75, 1.7500001
    rows[4, :16] = torch.arange(16, device="cuda") / 16 + 16  # ties between codes
    rows[4, 16] = 448
    rows[5, :] = 2.0 ** -130
    rows[6, 0], rows[6, 1] = -448 * 2.0 ** 100, 2.0 ** 90
    rows[7, :] = float("nan")
    codes = Codes(gpu_lib, 8, 256)
    gpu_lib.muon_ckpt_save(mat(rows, F32), codes.ck)
    unit, sb = T.checkpoint(n64(rows))
    got, gb = codes.read()
    assert np.array_equal(gb, sb) and np.array_equal(got, unit, equal_nan=True)
    back = out_mat(8, 256, F32)
    gpu_lib.muon_ckpt_load(codes.ck, back)
    with np.errstate(over="ignore"):  # the largest floats round up to the code of 2^128, an infinity in float32
        assert np.array_equal(n64(back), T.values(unit, sb).astype(np.float32), equal_nan=True)
    _, bf = padded(8, 256, BF)
    gpu_lib.muon_ckpt_load(codes.ck, bf)
    assert torch.equal(torch.nan_to_num(bf, nan=7.0), torch.nan_to_num(back.to(BF), nan=7.0))
    none = gpu_lib.Checkpoint.empty(0, 70)
    gpu_lib.muon_ckpt_save(torch.empty((0, 70), device="cuda"), none)


def saved(mu, x):
    ck = mu.Checkpoint.empty(*x.shape)
    mu.muon_ckpt_save(x, ck)
    back = torch.empty(x.shape, device="cuda")
    mu.muon_ckpt_load(ck, back)
    return ck, n64(back)


def wgrad_tol(dtype, ref, mag, length):
    # sums of 16 products in the matrix core, one after another; three parts of a float32 gradient
    return HALF[dtype] * np.abs(ref) + (length / 4 + 40) * U * mag


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("slots,n,k,extra", [(1, 1, 1, 0), (1, 3, 5, 0), (31, 64, 64, 0), (32, 128, 256, 0), (33, 130, 260, 0),
                                             (65, 127, 255, 1), (200, 7, 513, 0), (97, 300, 129, 3), (1500, 136, 272, 0),
                                             (4000, 64, 70, 0)])
def test_weight_grad_dense(gpu_lib, slots, n, k, extra, dtype):
    mu, g = gpu_lib, gen(slots * 7 + n)
    ck, X = saved(mu, randn(g, slots, k) * torch.exp(randn(g, 1, k)))
    dy = mat(randn(g, slots, n, scale=1e-3), dtype, extra)
    out = out_mat(n, k, dtype, extra)
    mu.muon_ckpt_weight_grad(dy, ck, out[None])
    ref, mag = T.weight_grad(n64(dy), X)
    close(n64(out), ref[0], wgrad_tol(dtype, ref[0], mag[0], slots), "gradient")


def lists(g, tokens, topk, experts, seed_popular=1.0):
    want = randn(g, experts) * seed_popular + randn(g, tokens, experts)
    picked = want.topk(topk, 1).indices.reshape(-1)
    rows = torch.argsort(picked, stable=True).to(torch.int32)
    counts = torch.bincount(picked, minlength=experts)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    return rows, offsets


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("tokens,topk,experts,n,k", [(1, 1, 2, 5, 9), (3, 3, 7, 66, 131), (100, 8, 16, 64, 260),
                                                     (333, 5, 40, 129, 64), (700, 2, 3, 768, 300)])
def test_weight_grad_groups(gpu_lib, tokens, topk, experts, n, k, dtype):
    mu, g = gpu_lib, gen(tokens + experts)
    ck, X = saved(mu, randn(g, tokens, k))
    rows, offsets = lists(g, tokens, topk, experts, 2.0)
    dy = mat(randn(g, tokens * topk, n, scale=1e-3), dtype)
    out = out_mat(experts * n, k, dtype)
    mu.muon_ckpt_weight_grad(dy, ck, out.view(experts, n, k), offsets, rows, topk)
    ref, mag = T.weight_grad(n64(dy), X, offsets.tolist(), rows.cpu().numpy(), topk)
    length = int((offsets[1:] - offsets[:-1]).max())
    close(n64(out).reshape(ref.shape), ref, wgrad_tol(dtype, ref, mag, length), "gradients")


def test_weight_grad_odd_lists(gpu_lib):
    """Empty groups, slots of no token, offsets beyond the slots, no slots at all; a float32 gradient's infinities."""
    mu, g = gpu_lib, gen(3)
    ck, X = saved(mu, randn(g, 10, 40))
    dy = mat(randn(g, 12, 20), F32)
    rows = torch.tensor([0, 3, -1, 7, 9, 10, 400, 2, 2, 1, 5, 6], dtype=torch.int32, device="cuda")
    offsets = torch.tensor([-5, 0, 4, 4, 9, 70], dtype=torch.int32, device="cuda")
    out = out_mat(5 * 20, 40, F32).view(5, 20, 40)
    mu.muon_ckpt_weight_grad(dy, ck, out, offsets, rows, 1)
    there = (rows >= 0) & (rows < 10)
    D = n64(dy) * there.cpu().numpy()[:, None]
    ref, mag = T.weight_grad(D, X, [0, 0, 4, 4, 9, 12], rows.clamp(0, 9).cpu().numpy(), 1)
    close(n64(out), ref, wgrad_tol(F32, ref, mag, 12), "gradients")
    empty = torch.empty((0, 20), device="cuda")
    mu.muon_ckpt_weight_grad(empty, ck, out, torch.zeros(6, dtype=torch.int32, device="cuda"),
                             torch.empty(0, dtype=torch.int32, device="cuda"), 1)
    assert not n64(out).any()
    dy[3, 2], dy[4, 5] = float("inf"), float("nan")
    one = out_mat(20, 40, F32)
    mu.muon_ckpt_weight_grad(dy, ck, one[None], rows=rows)
    assert bool(torch.isnan(one[5]).all()) and not bool(torch.isfinite(one[2]).any())
    assert bool(torch.isfinite(one[[0, 1, 3, 4]]).all()) and bool(torch.isfinite(one[6:]).all())
    assert bool((one[2][torch.from_numpy(X[7] > 0).cuda()] == float("inf")).all())


def test_weight_grad_keeps_float32(gpu_lib):
    """A float32 gradient reaches the sum whole: one slot, x a power of two."""
    ck, _ = saved(gpu_lib, torch.full((1, 8), 4.0, device="cuda"))
    dy = mat(randn(gen(8), 1, 500) * torch.exp(5 * randn(gen(9), 1, 500)), F32)
    out = out_mat(500, 8, F32)
    gpu_lib.muon_ckpt_weight_grad(dy, ck, out[None])
    assert torch.equal(out, (4 * dy).t().expand(500, 8))


def route_all(mu, logits, topk, **kw):
    tokens, experts = logits.shape
    i32 = dict(dtype=torch.int32, device="cuda")
    out = (torch.full((tokens, topk), 77, **i32), torch.full((tokens, topk), 7.0, device="cuda"),
           torch.full((experts + 1,), 77, **i32), torch.full((experts + 1,), 77, **i32),
           torch.full((tokens * topk,), 77, **i32), torch.full((1,), 7.0, device="cuda"))
    mu.muon_route_forward(logits, *out, **kw)
    return out


ROUTE = [(1, 1, 1), (1, 5, 2), (7, 64, 8), (128, 128, 8), (129, 65, 3), (1000, 384, 8), (300, 385, 1), (65, 1024, 32),
         (2500, 7, 7), (66000, 3, 1)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("tokens,experts,topk", ROUTE)
def test_route(gpu_lib, tokens, experts, topk, renorm, dtype):
    mu, g = gpu_lib, gen(tokens + experts)
    v = randn(g, tokens, experts) * 1.5
    if tokens > 4:
        v[tokens - tokens // 5:] = -float("inf")   # padding
        v[1, experts // 2:] = -float("inf")
        v[2] = 0.25                                 # ties
    logits = mat(v, dtype, 3)
    idx, w, counts, offs, rows, loss = route_all(mu, logits, topk, alpha=0.3, renormalize=renorm)
    L = n64(logits)
    ri, rw, rc, ro, rr, rl = T.route(L, topk, 0.3, renorm)
    for got, ref in ((idx, ri), (counts, rc), (offs, ro), (rows, rr)):
        assert np.array_equal(got.cpu().numpy(), ref)
    spread = np.nanmax(np.where(np.isfinite(L), L, np.nan)) - np.nanmin(np.where(np.isfinite(L), L, np.nan))
    # the exponent's argument is rounded, sums of 16 registers over 64 lanes
    rel = (24 + spread) * 2 * U
    close(n64(w), rw, rel * rw, "weights")
    close(n64(loss)[0], rl, (rel + 128 * U) * abs(rl), "loss")
    dw = randn(g, tokens, topk)
    dloss = torch.full((1,), 0.7, device="cuda")
    dl = out_mat(tokens, experts, dtype, 3)
    mu.muon_route_backward(logits, idx, counts, dl, dweights=dw, dloss=dloss, alpha=0.3, renormalize=renorm)
    a, dl7 = float(np.float32(0.3)), float(np.float32(0.7))
    ref = T.route_grad(L, ri, rc, topk, n64(dw), dl7, a, renorm)
    p = T.softmax(L)
    d = np.tile(dl7 * a * experts / (topk * max(1, int(rc[-1])) ** 2) * rc[:-1], (tokens, 1))
    extra = np.zeros_like(p)
    safe = np.maximum(ri, 0)
    gw = np.where(ri >= 0, np.abs(n64(dw)), 0)
    if renorm:
        q = np.where(ri >= 0, np.take_along_axis(p, safe, 1), 0)
        q = q / np.maximum(q.sum(1, keepdims=True), 1e-300)
        gw = q * (gw + (q * gw).sum(1, keepdims=True))
        np.put_along_axis(extra, safe, np.maximum(gw, np.take_along_axis(extra, safe, 1)), 1)
    else:
        np.put_along_axis(extra, safe, np.maximum(gw, np.take_along_axis(extra, safe, 1)), 1)
        d, extra = d + extra, 0 * extra
    mag = p * (d + (d * p).sum(1, keepdims=True)) + extra
    tiny = 2.0 ** -133 if dtype == BF else 2.0 ** -149  # below the normal range a step is absolute
    close(n64(dl), ref, HALF[dtype] * np.abs(ref) + 3 * rel * mag + tiny, "dlogits")


def test_route_backward_is_the_slope(gpu_lib):
    """The gradient against differences of the forward pass's own weights and loss, in float32: steps of 2^-6 leave
    truncation near h^2 / 6 of third derivatives (at most 1) and rounding near 8 u / h."""
    mu, g = gpu_lib, gen(12)
    tokens, experts, topk, h = 4, 9, 3, 2.0 ** -6
    v = torch.sort(randn(g, tokens, experts), 1).values + torch.arange(experts, device="cuda") * 0.2  # no choice changes
    logits = mat(v, F32)
    dw = randn(g, tokens, topk)
    for renorm in (True, False):
        idx, w, counts, _, _, _ = route_all(mu, logits, topk, alpha=0.5, renormalize=renorm)
        dl = out_mat(tokens, experts, F32)
        mu.muon_route_backward(logits, idx, counts, dl, dweights=dw, dloss=torch.ones(1, device="cuda"), alpha=0.5,
                               renormalize=renorm)
        for t in range(tokens):
            for e in range(experts):
                f = []
                for s in (h, -h):
                    moved = logits.clone()
                    moved[t, e] += s
                    i2, w2, _, _, _, l2 = route_all(mu, moved, topk, alpha=0.5, renormalize=renorm)
                    assert torch.equal(i2, idx)
                    f.append(float(l2.double() + (w2.double() * dw.double()).sum()))
                slope = (f[0] - f[1]) / (2 * h)
                assert abs(float(dl[t, e]) - slope) <= 10 * (h * h / 6 + 8 * U / h), (renorm, t, e)


def test_route_masked_everywhere_and_empty(gpu_lib):
    mu = gpu_lib
    logits = mat(torch.full((200, 10), -float("inf"), device="cuda"), BF)
    idx, w, counts, offs, rows, loss = route_all(mu, logits, 4)
    assert bool((idx == -1).all() and (w == 0).all() and (counts == 0).all() and (offs == 0).all() and (rows == -1).all())
    assert float(loss) == 0
    dl = out_mat(200, 10, BF)
    mu.muon_route_backward(logits, idx, counts, dl, dweights=torch.ones((200, 4), device="cuda"), dloss=torch.ones(1, device="cuda"))
    assert not n64(dl).any()
    none = torch.empty((0, 10), device="cuda")
    idx, w, counts, offs, rows, loss = route_all(mu, none, 4)
    assert not n64(counts).any() and not n64(offs).any() and float(loss) == 0
    # the lowest finite value is a logit like any other; NaN and infinities end nothing and stay in range
    low = torch.full((3, 6), torch.finfo(F32).min, device="cuda")
    low[1, 2], low[2, 4] = float("nan"), float("inf")
    idx, w, counts, offs, rows, loss = route_all(mu, low, 2)
    assert idx.tolist() == [[0, 1], [0, 1], [4, 0]] and int(counts[6]) == 3
    assert bool(torch.isnan(w[1]).all()) and np.allclose(n64(w[0]), 0.5)


def test_same_bits_every_time_and_on_other_streams(gpu_lib):
    """Two runs of every operator on different streams give the same bits, and what the thread had set stays set."""
    import ctypes
    mu, g = gpu_lib, gen(21)
    keep = torch.empty(4096, dtype=torch.uint8, device="cuda")
    mu.muon_set_workspace(keep.data_ptr(), 4096)
    tokens, experts, topk, n, k = 700, 12, 3, 96, 640
    x = randn(g, tokens, k).to(BF)
    dy = randn(g, tokens * topk, n).to(BF)
    dn = randn(g, tokens, k).to(BF)
    logits = randn(g, tokens, experts)
    w, b = randn(g, 1, k).to(BF), randn(g, 1, k).to(BF)
    dw = randn(g, tokens, topk)
    torch.cuda.synchronize()

    def all_of_it():
        y, dx, ck = torch.empty_like(x), torch.empty_like(x), mu.Checkpoint.empty(tokens, k)
        mean, rstd = torch.empty(tokens, device="cuda"), torch.empty(tokens, device="cuda")
        mu.muon_layernorm_forward(x, y, mean, rstd, w, b, ckpt=ck)
        r = route_all(mu, logits, topk)
        grads = torch.empty((experts, n, k), dtype=BF, device="cuda")
        mu.muon_ckpt_weight_grad(dy, ck, grads, r[3], r[4], topk)
        dl, gw, gb = torch.empty_like(logits), torch.empty_like(w), torch.empty_like(b)
        mu.muon_route_backward(logits, r[0], r[2], dl, dweights=dw, dloss=r[5])
        mu.muon_layernorm_backward(dn, x, mean, rstd, dx, w, gw, gb)
        return [y, mean, rstd, ck.codes.view(torch.uint8).clone(), ck.scales, grads, dl, dx, gw, gb, *r]

    first = all_of_it()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        second = all_of_it()
    torch.cuda.synchronize()
    for p, q in zip(first, second):
        assert torch.equal(p, q)
    ptr, size = ctypes.c_void_p(), ctypes.c_size_t()
    assert mu.lib().muon_get_workspace(ctypes.byref(ptr), ctypes.byref(size)) == 0
    assert ptr.value == keep.data_ptr() and size.value == 4096
    mu.muon_set_workspace(None, 0)
    mu.muon_set_stream(None)


def test_graph_replays(gpu_lib):
    """Captured once with the caller's workspace, replayed on new inputs with eager work between, equal to eager calls."""
    mu, g = gpu_lib, gen(22)
    tokens, experts, topk, n, k = 300, 8, 2, 80, 384
    x, dn = torch.empty((tokens, k), dtype=BF, device="cuda"), torch.empty((tokens, k), dtype=BF, device="cuda")
    dy, logits = torch.empty((tokens * topk, n), device="cuda"), torch.empty((tokens, experts), device="cuda")
    w = randn(g, 1, k).to(BF)
    size = max(mu.muon_layernorm_workspace_size(tokens, k), mu.muon_route_workspace_size(tokens, experts, topk),
               mu.muon_ckpt_weight_grad_workspace_size(mu.MUON_F32, tokens * topk, n, k, experts), 256)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")

    def make():
        return dict(y=torch.empty_like(x), dx=torch.empty_like(x), mean=torch.empty(tokens, device="cuda"),
                    rstd=torch.empty(tokens, device="cuda"), ck=mu.Checkpoint.empty(tokens, k),
                    idx=torch.empty((tokens, topk), **i32), wt=torch.empty((tokens, topk), device="cuda"),
                    counts=torch.empty(experts + 1, **i32), offs=torch.empty(experts + 1, **i32),
                    rows=torch.empty(tokens * topk, **i32), loss=torch.empty(1, device="cuda"),
                    grads=torch.empty((experts, n, k), device="cuda"), dl=torch.empty_like(logits), gw=torch.empty_like(w))

    def step(o):
        mu.muon_layernorm_forward(x, o["y"], o["mean"], o["rstd"], w, ckpt=o["ck"])
        mu.muon_route_forward(logits, o["idx"], o["wt"], o["counts"], o["offs"], o["rows"], o["loss"], workspace=ws)
        mu.muon_ckpt_weight_grad(dy, o["ck"], o["grads"], o["offs"], o["rows"], topk, workspace=ws)
        mu.muon_route_backward(logits, o["idx"], o["counts"], o["dl"], dloss=o["loss"])
        mu.muon_layernorm_backward(dn, x, o["mean"], o["rstd"], o["dx"], w, o["gw"], workspace=ws)

    def fill(seed):
        h = gen(seed)
        for t in (x, dn, dy, logits):
            t.copy_(randn(h, *t.shape))

    captured, eager = make(), make()
    fill(1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(captured)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step(captured)
    torch.cuda.synchronize()
    for seed in (1, 2, 3):
        fill(seed)
        step(eager)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for name in eager:
            if name != "ck":
                assert torch.equal(captured[name], eager[name]), (seed, name)
    mu.muon_set_stream(None)


def test_layernorm_of_more_rows_than_one_launch(gpu_lib):
    """Past 2^32 threads' worth of rows: the last ones are those of a call on them alone."""
    rows, cols = (1 << 23) + 5, 8
    x = torch.empty((rows, cols), dtype=BF, device="cuda").normal_(generator=gen(31))
    y, mean, rstd = torch.empty_like(x), torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    gpu_lib.muon_layernorm_forward(x, y, mean, rstd)
    for part in (slice(0, 1000), slice((1 << 23) - 500, (1 << 23) + 5)):
        y2, m2, r2 = torch.empty_like(x[part]), mean[part].clone(), rstd[part].clone()
        gpu_lib.muon_layernorm_forward(x[part], y2, m2, r2)
        assert torch.equal(y2, y[part]) and torch.equal(m2, mean[part]) and torch.equal(r2, rstd[part])
        close(n64(y2), T.layernorm(n64(x[part]))[0], 2.0 ** -8 * np.abs(n64(y2)) + 2e-3, "y")


def test_weight_grad_of_one_slot_into_many_groups(gpu_lib):
    """Buffers smaller than a run, through the element form: the one slot belongs to group 2 of 40."""
    ck, X = saved(gpu_lib, torch.tensor([[1.5, -2.0, 3.0]], device="cuda"))
    dy = mat(torch.tensor([[0.5, 4.0]], device="cuda"), F32)
    offsets = torch.tensor([0, 0, 0] + [1] * 38, dtype=torch.int32, device="cuda")
    out = out_mat(40 * 2, 3, F32).view(40, 2, 3)
    gpu_lib.muon_ckpt_weight_grad(dy, ck, out, offsets, torch.zeros(1, dtype=torch.int32, device="cuda"))
    ref, _ = T.weight_grad(n64(dy), X, offsets.tolist(), [0])
    assert np.array_equal(n64(out), ref)  # exact in float32


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("tokens,topk,experts,n,k", [(1600, 2, 3, 129, 131), (900, 1, 1, 300, 515), (2500, 4, 8, 64, 48)])
def test_weight_grad_long_groups(gpu_lib, tokens, topk, experts, n, k, dtype):
    """Groups long enough for the wider form, through their lists, with slots of no token among them."""
    mu, g = gpu_lib, gen(tokens + n)
    ck, X = saved(mu, randn(g, tokens, k))
    rows, offsets = lists(g, tokens, topk, experts)
    dy = mat(randn(g, tokens * topk, n, scale=1e-3), dtype)
    gone = torch.rand(len(rows), generator=g, device="cuda") < 0.01
    bad = torch.where(torch.arange(len(rows), device="cuda") % 2 == 0, -1, tokens * topk).to(torch.int32)
    rows = torch.where(gone, bad, rows)
    dy[gone] = float("nan")  # what such a slot's gradient holds does not count
    out = out_mat(experts * n, k, dtype)
    mu.muon_ckpt_weight_grad(dy, ck, out.view(experts, n, k), offsets, rows, topk)
    there = torch.where(gone, 0, rows)
    D = np.where(gone.cpu().numpy()[:, None], 0.0, n64(dy))
    ref, mag = T.weight_grad(D, X, offsets.tolist(), there.cpu().numpy(), topk)
    length = int((offsets[1:] - offsets[:-1]).max())
    close(n64(out).reshape(ref.shape), ref, wgrad_tol(dtype, ref, mag, length), "gradients")


@pytest.mark.parametrize("dtype", [BF, F32])
def test_weight_grad_of_more_tiles_than_run_at_once(gpu_lib, dtype):
    """Groups by length: very uneven, equal and empty ones, and slots outside every group."""
    mu, g = gpu_lib, gen(41)
    tokens, n, k = 900, 256, 2304
    counts = [700, 0, 500, 700, 3, 1, 0, 500] * 4
    slots = sum(counts) + 9
    ck, X = saved(mu, randn(g, tokens, k))
    rows = torch.randint(0, tokens, (slots,), generator=g, device="cuda").to(torch.int32)
    offsets = torch.tensor(np.append(0, np.cumsum(counts)), dtype=torch.int32, device="cuda")
    dy = mat(randn(g, slots, n, scale=1e-3), dtype)
    out = out_mat(len(counts) * n, k, dtype)
    assert mu.muon_ckpt_weight_grad_workspace_size(mu.MUON_F32 if dtype == F32 else mu.MUON_BF16, slots, n, k, len(counts)) > 0
    mu.muon_ckpt_weight_grad(dy, ck, out.view(len(counts), n, k), offsets, rows)
    ref, mag = T.weight_grad(n64(dy), X, offsets.tolist(), rows.cpu().numpy())
    close(n64(out).reshape(ref.shape), ref, wgrad_tol(dtype, ref, mag, max(counts)), "gradients")


@pytest.mark.parametrize("slots", [3, 40])
def test_weight_grad_of_slots_below_zero(gpu_lib, slots):
    """A negative slot has no token, however many slots a token has: both for buffers smaller than a run and through the tiles."""
    mu, g = gpu_lib, gen(51)
    ck, X = saved(mu, randn(g, 3, 40))
    dy = mat(randn(g, slots, 2), F32)
    rows = torch.tensor([-1, 0, -7] + [-(1 << 31)] * (slots - 3), dtype=torch.int32, device="cuda")
    for per in ((1 << 31) - 1, 1 << 30, 1):
        out = out_mat(2, 40, F32)
        mu.muon_ckpt_weight_grad(dy, ck, out[None], rows=rows, rows_per_token=per)
        ref, mag = T.weight_grad(n64(dy)[1:2], X, [0, 1], [0])
        close(n64(out), ref[0], wgrad_tol(F32, ref[0], mag[0], 3), "gradient")


@pytest.mark.parametrize("dtype", [BF, F32])
def test_weight_grad_slots_of_no_token_beside_any_checkpoint(gpu_lib, dtype):
    """What lies in a token's codes and scales does not reach a sum that has no slot of it."""
    mu, g = gpu_lib, gen(52)
    ck, X = saved(mu, randn(g, 50, 200))
    ck.codes.view(torch.uint8)[0] = 0x7F
    rows = torch.arange(1, 41, device="cuda", dtype=torch.int32)
    rows[::3] = -1
    dy = mat(randn(g, 40, 24, scale=1e-3), dtype)
    there = (rows > 0).cpu().numpy()
    ref, mag = T.weight_grad(n64(dy)[there], X, [0, int(there.sum())], rows.cpu().numpy()[there])
    for byte in (0, 247, 248, 254, 255):
        ck.scales[0] = byte
        out = out_mat(24, 200, dtype)
        mu.muon_ckpt_weight_grad(dy, ck, out[None], rows=rows)
        close(n64(out), ref[0], wgrad_tol(dtype, ref[0], mag[0], 40), f"gradient, scale byte {byte}")


def test_checkpoint_whose_memory_was_exchanged(gpu_lib):
    """A save, a load and a weight gradient after the tensors' memory has been exchanged use the new memory."""
    mu, g = gpu_lib, gen(53)
    ck, _ = saved(mu, randn(g, 20, 256))
    held = ck.codes.data, ck.scales.data
    before = [t.view(torch.uint8).clone() for t in held]
    ck.codes.data, ck.scales.data = torch.zeros_like(held[0]), torch.zeros_like(held[1])
    x = randn(g, 20, 256)
    mu.muon_ckpt_save(x, ck)
    assert all(torch.equal(t.view(torch.uint8), b) for t, b in zip(held, before))
    unit, sb = T.checkpoint(n64(x))
    back = out_mat(20, 256, F32)
    mu.muon_ckpt_load(ck, back)
    X = T.values(unit, sb)
    assert np.array_equal(n64(back), X)
    dy, out = mat(randn(g, 20, 9), F32), out_mat(9, 256, F32)
    mu.muon_ckpt_weight_grad(dy, ck, out[None])
    ref, mag = T.weight_grad(n64(dy), X)
    close(n64(out), ref[0], wgrad_tol(F32, ref[0], mag[0], 20), "gradient")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("cols,early,waves,runs", [(1024, 512, 1, 2), (7168, 2048, 4, 4), (32768, 8192, 16, 4)])
def test_layernorm_variance_is_no_chain(gpu_lib, cols, early, waves, runs, dtype):
    """Each thread's first value is 1, and its others' squares lie just under the half step that adding them to 1 one by
    one would lose. Neighbours are negatives of each other, so the mean is 0 exactly. A tree over a run of eight and over
    the runs, then equal sums of the lanes (doublings, exact) and of the waves in turn; a square, a division, half of that
    in rstd, its root and reciprocal."""
    v = torch.full((3, cols), 2.0 ** -12 * 255 / 256, device="cuda")
    v[:, :early:8] = 1
    v[:, 8::16] *= -1
    for i in range(1, 8):
        v[:, i::16] *= (-1) ** i
        v[:, 8 + i::16] *= -(-1) ** i
    x, y = mat(v, dtype), out_mat(3, cols, dtype)
    mean, rstd = torch.empty(3, device="cuda"), torch.empty(3, device="cuda")
    gpu_lib.muon_layernorm_forward(x, y, mean, rstd, eps=0.0)
    _, _, ref = T.layernorm(n64(x), eps=0.0)
    assert not n64(mean).any()
    levels = 3 + int(np.log2(runs)) + waves - 1
    close(n64(rstd), ref, ((levels + 2) / 2 + 2) * U * ref, "rstd")


def test_layernorm_gradient_sums_are_no_chain(gpu_lib):
    """Each slice of the workgroups' partial sums starts with a 1 and goes on with values just under the half step that
    adding them to it one by one would lose (167 workgroups of rows b and b + 167, eight slices). A row sum, a tree over
    eight partials, three such groups in turn, eight slices, the result."""
    mu, g = gpu_lib, gen(54)
    rows, cols, blocks = 333, 2047, 167
    dy = torch.zeros((rows, cols), device="cuda")
    dy[:blocks] = 2.0 ** -24 * 255 / 256
    dy[:8] = 1
    x = randn(g, rows, cols).sign()  # mean 0 and rstd 1, as passed: dweight is the same sum but for the signs
    x[:, ::2] = 1
    dy, x, dx = mat(dy, F32), mat(x, F32), out_mat(rows, cols, F32)
    mean, rstd = torch.zeros(rows, device="cuda"), torch.ones(rows, device="cuda")
    dw, db = out_mat(1, cols, F32), out_mat(1, cols, F32)
    mu.muon_layernorm_backward(dy, x, mean, rstd, dx, None, dw, db)
    _, rdw, rdb = T.layernorm_grad(n64(dy), n64(x), n64(mean), n64(rstd))
    tol = (1 + 3 + 2 + 3 + 1) * U * np.abs(n64(dy)).sum(0)
    close(n64(db)[0], rdb, tol, "dbias")
    close(n64(dw)[0], rdw, tol, "dweight")


@pytest.mark.parametrize("wdtype", [BF, F32])
def test_layernorm_infinite_weight_and_bias(gpu_lib, wdtype):
    """An infinite weight makes its column infinite, with the sign of x - mean, and no other."""
    mu, g = gpu_lib, gen(56)
    x = mat(randn(g, 5, 300), F32)
    w, b = mat(torch.ones((1, 300), device="cuda"), wdtype), mat(torch.zeros((1, 300), device="cuda"), wdtype)
    w[0, 3], w[0, 4], w[0, 5], b[0, 6], b[0, 7] = float("inf"), -float("inf"), float("nan"), -float("inf"), float("nan")
    y, z = out_mat(5, 300, F32), out_mat(5, 300, F32)
    mu.muon_layernorm_forward(x, y, weight=w, bias=b)
    mu.muon_layernorm_forward(x, z)
    inf = torch.full((5,), float("inf"), device="cuda")
    assert torch.equal(y[:, 3], torch.copysign(inf, z[:, 3])) and torch.equal(y[:, 4], torch.copysign(inf, -z[:, 4]))
    assert bool(torch.isnan(y[:, 5]).all()) and torch.equal(y[:, 6], -inf) and bool(torch.isnan(y[:, 7]).all())
    assert torch.equal(y[:, 8:], z[:, 8:]) and torch.equal(y[:, :3], z[:, :3])


@pytest.mark.parametrize("cols", [1, 7, 300, 7168, 20000])
def test_layernorm_of_equal_values(gpu_lib, cols):
    """A row of equal bf16 values has their mean exactly, variance 0 and the bias as its output."""
    v = torch.tensor([[0.0], [1.0], [-0.1], [300.0], [3e-5]], device="cuda").to(BF)
    x, b = mat(v.expand(5, cols), BF), mat(randn(gen(57), 1, cols), BF)
    y, mean, rstd = out_mat(5, cols, BF), torch.empty(5, device="cuda"), torch.empty(5, device="cuda")
    gpu_lib.muon_layernorm_forward(x, y, mean, rstd, None, b, eps=2.0 ** -16)
    assert torch.equal(mean, v[:, 0].float()) and bool((rstd == 256).all())
    assert torch.equal(y, b.expand(5, cols))


def check_groups(mu, dy, ck, X, out, offsets=None, rows=None, topk=1):
    """All elements of the groups' gradients against 64-bit products on the GPU."""
    X = torch.from_numpy(X).cuda()
    ends = [0, dy.shape[0]] if offsets is None else offsets.tolist()
    for i in range(len(ends) - 1):
        s = torch.arange(ends[i], ends[i + 1], device="cuda")
        x = X[torch.div(s if rows is None else rows[s].long(), topk, rounding_mode="floor")]
        d = dy[s].double()
        ref, mag = torch.mm(d.t(), x), torch.mm(d.abs().t(), x.abs())
        tol = HALF[dy.dtype] * ref.abs() + (len(s) / 4 + 40) * U * mag  # as wgrad_tol
        bad = ~((out[i].double() - ref).abs() <= tol)
        assert not bool(bad.any()), f"group {i} of {len(s)} slots: {int(bad.sum())} off"


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("listed", [False, True])
def test_weight_grad_of_long_sums_into_many_tiles(gpu_lib, listed, dtype):
    """One group of 1000 slots into 17 x 17 tiles: four waves a tile and no partial sums, with and without a list."""
    mu, g = gpu_lib, gen(61)
    slots, n, k = 1000, 2050, 4100
    assert mu.muon_ckpt_weight_grad_workspace_size(mu.MUON_F32 if dtype == F32 else mu.MUON_BF16, slots, n, k) == 0
    ck, X = saved(mu, randn(g, slots, k) * torch.exp(randn(g, 1, k)))
    dy, out = mat(randn(g, slots, n, scale=1e-3), dtype, 3), out_mat(n, k, dtype)
    rows = torch.randperm(slots, generator=g, device="cuda").to(torch.int32) if listed else None
    mu.muon_ckpt_weight_grad(dy, ck, out[None], rows=rows)
    check_groups(mu, dy, ck, X, out[None], rows=rows)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,k,counts,ordered", [(1030, 2570, [1100, 31, 1300], False),
                                                (2050, 1300, [2500, 0, 33, 900, 1200, 700], True)])
def test_weight_grad_of_long_uneven_groups(gpu_lib, n, k, counts, ordered, dtype):
    """768 slots a group and more on average: four waves a tile and no partial sums, in the given order and the longest first."""
    mu, g = gpu_lib, gen(62)
    slots, topk = sum(counts), 3
    tokens = -(-slots // topk)
    size = mu.muon_ckpt_weight_grad_workspace_size(mu.MUON_F32 if dtype == F32 else mu.MUON_BF16, slots, n, k, len(counts))
    assert size == (16 * len(counts) if ordered else 0)
    ck, X = saved(mu, randn(g, tokens, k))
    rows = torch.randperm(tokens * topk, generator=g, device="cuda")[:slots].to(torch.int32)
    offsets = torch.tensor(np.append(0, np.cumsum(counts)), dtype=torch.int32, device="cuda")
    dy, out = mat(randn(g, slots, n, scale=1e-3), dtype), out_mat(len(counts) * n, k, dtype)
    mu.muon_ckpt_weight_grad(dy, ck, out.view(len(counts), n, k), offsets, rows, topk)
    check_groups(mu, dy, ck, X, out.view(len(counts), n, k), offsets, rows, topk)


@pytest.mark.parametrize("dtype,wdtype", [(BF, BF), (BF, F32), (F32, F32), (F32, BF)])
@pytest.mark.parametrize("rows,cols,extra", [(515, 9000, 0), (700, 12287, 1), (520, 20001, 3), (515, 32768, 0)])
def test_layernorm_wide_rows_of_several_to_a_workgroup(gpu_lib, rows, cols, extra, dtype, wdtype):
    test_layernorm(gpu_lib, rows, cols, extra, dtype, wdtype)


def test_buffers_that_interleave_without_overlap(gpu_lib):
    """Operands whose rows lie between each other's are no overlap; one byte further they are."""
    mu, g = gpu_lib, gen(63)
    rows, cols = 37, 300
    wide = torch.zeros((rows, 2 * cols), dtype=BF, device="cuda")
    x, y = wide[:, :cols], wide[:, cols:]
    x.copy_(randn(g, rows, cols))
    want = torch.empty((rows, cols), dtype=BF, device="cuda")
    mu.muon_layernorm_forward(x.clone(), want)
    before = x.clone()
    mu.muon_layernorm_forward(x, y)
    assert torch.equal(y, want) and torch.equal(x, before)
    with pytest.raises(mu.MuonError) as e:
        mu.muon_layernorm_forward(x, wide[:, cols - 1:2 * cols - 1])
    assert e.value.status == mu.MUON_ERR_ALIAS
    # a row of values, then its codes, then its scales
    buf = torch.zeros((rows, 3 * cols + 4), dtype=torch.uint8, device="cuda")
    v = buf.view(BF)[:, :cols]
    v.copy_(randn(g, rows, cols))
    kept = v.clone()
    ck = mu.Checkpoint(buf[:, 2 * cols:3 * cols].view(torch.float8_e4m3fn), buf[:, 3 * cols:3 * cols + 3])
    mu.muon_ckpt_save(v, ck)
    other = mu.Checkpoint.empty(rows, cols)
    mu.muon_ckpt_save(kept, other)
    assert torch.equal(v, kept) and torch.equal(ck.scales, other.scales) and not bool(buf[:, 3 * cols + 3].any())
    assert torch.equal(ck.codes.view(torch.uint8), other.codes.view(torch.uint8))
    with pytest.raises(mu.MuonError) as e:
        mu.muon_ckpt_save(v, mu.Checkpoint(buf[:, 2 * cols - 1:3 * cols - 1].view(torch.float8_e4m3fn), buf[:, 3 * cols:3 * cols + 3]))
    assert e.value.status == mu.MUON_ERR_ALIAS


def test_layernorm_codes_near_their_borders(gpu_lib):
    """8-bit codes of the output that differ from those of the exact output (in 64 bits, as float32, rounded to bf16). One
    does where a border between two codes lies between both: borders are 2^-4 to 2^-3 apart, so that a result a quarter
    of a unit of 2^-24 off passes one in 2^-22 of cases; and where such a result rounds to another float32 value, a
    quarter of cases, one of 2^20 patterns decides on either side, 2^-21. A result with three float32 roundings is off by
    half a unit or more, and has twice as many."""
    mu, g = gpu_lib, gen(58)
    rows, cols = 8192, 7168
    spread = torch.exp(0.5 * randn(g, cols))
    spread[::250] *= 20
    x = (randn(g, rows, cols) * spread + 0.3 * randn(g, cols)).to(BF)
    w, b = (1 + 0.2 * randn(g, 1, cols)).to(BF), (0.1 * randn(g, 1, cols)).to(BF)
    y, ck, want = torch.empty_like(x), mu.Checkpoint.empty(rows, cols), mu.Checkpoint.empty(rows, cols)
    mu.muon_layernorm_forward(x, y, None, None, w, b, ckpt=ck)
    X = x.double()
    var, mean = torch.var_mean(X, 1, correction=0, keepdim=True)
    ref = (X - mean) / (var + float(np.float32(1e-5))).sqrt() * w.double() + b.double()
    mu.muon_ckpt_save(ref.float().to(BF), want)
    off = int((ck.codes.view(torch.uint8) != want.codes.view(torch.uint8)).sum())
    assert off <= rows * cols * (2.0 ** -22 + 2.0 ** -21), off
    # the same bits without a checkpoint
    z = torch.empty_like(y)
    mu.muon_layernorm_forward(x, z, None, None, w, b)
    assert torch.equal(y, z)
