"""Plain float64 oracles of the training operators: layer norm, 8-bit
activation checkpoints, expert weight gradients, routing.

TEST INFRASTRUCTURE ONLY; the library never calls it and shares no code with
it. Layer norm: Ba, Kiros and Hinton, "Layer Normalization", over the columns
of each row. Checkpoint codes: the OCP 8-bit floating point format E4M3 (four
exponent bits of bias 7, three fraction bits, largest 448, no infinities)
with one power-of-two scale per group of columns. Balance loss: Fedus, Zoph
and Shazeer, "Switch Transformers", section 2.2, for k choices a token.
"""
import numpy as np

GROUP = 128


def layernorm(x, weight=None, bias=None, eps=1e-5):
    """(y, mean, rstd)"""
    x = np.asarray(x, np.float64)
    mean = x.mean(1)
    xc = x - mean[:, None]
    rstd = 1 / np.sqrt((xc * xc).mean(1) + eps)
    y = xc * rstd[:, None]
    if weight is not None:
        y = y * weight
    return (y if bias is None else y + bias), mean, rstd


def layernorm_grad(dy, x, mean, rstd, weight=None):
    """(dx, dweight, dbias)"""
    xh = (x - mean[:, None]) * rstd[:, None]
    h = dy if weight is None else dy * weight
    dx = rstd[:, None] * (h - h.mean(1, keepdims=True) - xh * (h * xh).mean(1, keepdims=True))
    return dx, (dy * xh).sum(0), dy.sum(0)


def code_values():
    """What each of the 256 code bytes stands for."""
    b = np.arange(256)
    power, frac = (b >> 3) & 15, (b & 7) / 8.0
    v = np.where(power > 0, (1 + frac) * 2.0 ** (power - 7), frac * 2.0 ** -6)
    v[(b & 127) == 127] = np.nan
    return np.where(b > 127, -v, v)


def checkpoint(x):
    """(values on the code grid before scaling, scale bytes) of x's rows."""
    x = np.asarray(x, np.float64)
    rows, cols = x.shape
    groups = -(-cols // GROUP)
    unit, scales = np.empty_like(x), np.empty((rows, groups), np.int64)
    grid = np.sort(code_values()[:127])  # 0 .. 448
    for g in range(groups):
        part = x[:, g * GROUP:(g + 1) * GROUP]
        amax = np.where(np.isfinite(part), np.abs(part), 0).max(1)
        b = np.zeros(rows, np.int64)
        while np.any(amax > 448 * 2.0 ** (b - 127)):
            b = np.where(amax > 448 * 2.0 ** (b - 127), b + 1, b)
        scales[:, g] = b
        v = part / 2.0 ** (b - 127)[:, None]
        # nearest grid value, ties to the even code (codes 0 .. 126 ascend with their values)
        hi = np.clip(np.searchsorted(grid, np.abs(v)), 0, 126)
        lo = np.clip(hi - 1, 0, 126)
        with np.errstate(invalid="ignore"):
            dl, dh = np.abs(v) - grid[lo], grid[hi] - np.abs(v)
        code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
        unit[:, g * GROUP:(g + 1) * GROUP] = np.where(np.isfinite(v), np.copysign(grid[code], v), np.nan)
    return unit, scales


def values(unit, scales):
    rows, cols = unit.shape
    return unit * np.repeat(2.0 ** (np.asarray(scales, np.float64) - 127), GROUP, 1)[:, :cols]


def weight_grad(dy, x, offsets=None, rows=None, per_token=1):
    """(gradients of every group, sums of the products' magnitudes)"""
    slots = dy.shape[0]
    offsets = [0, slots] if offsets is None else offsets
    rows = np.arange(slots) if rows is None else rows
    out = np.zeros((len(offsets) - 1, dy.shape[1], x.shape[1]))
    mag = np.zeros_like(out)
    for g in range(len(offsets) - 1):
        s = np.arange(offsets[g], offsets[g + 1])
        token = np.asarray(rows)[s] // per_token
        out[g] = dy[s].T @ x[token]
        mag[g] = np.abs(dy[s]).T @ np.abs(x[token])
    return out, mag


def softmax(x):
    x = np.asarray(x, np.float64)
    top = x.max(1, keepdims=True)
    e = np.exp(x - np.where(top == -np.inf, 0, top))
    s = e.sum(1, keepdims=True)
    return e / np.where(s == 0, 1, s)


def route(logits, topk, alpha=1e-2, renormalize=True):
    """(indices, weights, counts, offsets, rows, loss)"""
    x = np.asarray(logits, np.float64)
    tokens, experts = x.shape
    p = softmax(x)
    order = np.argsort(-x, axis=1, kind="stable")[:, :topk]
    there = np.take_along_axis(x, order, 1) > -np.inf
    indices = np.where(there, order, -1)
    weights = np.where(there, np.take_along_axis(p, order, 1), 0.0)
    if renormalize:
        share = weights.sum(1, keepdims=True)
        weights = weights / np.where(share == 0, 1, share)
    flat = indices.reshape(-1)
    counts = np.bincount(flat[flat >= 0], minlength=experts)
    rows = np.full(tokens * topk, -1)
    placed = np.concatenate([np.flatnonzero(flat == e) for e in range(experts)]) if tokens else flat
    rows[:len(placed)] = placed
    n = int((x > -np.inf).any(1).sum())
    some = max(n, 1)
    loss = alpha * experts / (topk * some) * (counts * p.sum(0) / some).sum()
    return (indices, weights, np.append(counts, n), np.append(0, np.cumsum(counts)), rows, loss)


def route_grad(logits, indices, counts, topk, dweights=None, dloss=0.0, alpha=1e-2, renormalize=True):
    p = softmax(logits)
    tokens, experts = p.shape
    n = max(int(counts[experts]), 1)
    d = np.tile(dloss * alpha * experts / (topk * n * n) * np.asarray(counts[:experts], np.float64), (tokens, 1))
    more = np.zeros_like(p)
    if dweights is not None:
        for t in range(tokens):
            at = indices[t][indices[t] >= 0]
            g = dweights[t][indices[t] >= 0]
            if renormalize:
                w = p[t, at] / p[t, at].sum() if len(at) else p[t, at]
                more[t, at] += w * (g - (w * g).sum())
            else:
                d[t, at] += g
    return p * (d - (d * p).sum(1, keepdims=True)) + more
