"""Pins of the training operators' oracles: gradients against central
differences of the forward formulas, the checkpoint's grid and scale rule
against closed forms, the slot lists against a direct search."""
import numpy as np
import pytest

from oracle import train_oracle as T


def central(f, x, h=1e-6):
    g = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        a, b = x.copy(), x.copy()
        a[i] += h
        b[i] -= h
        g[i] = (f(a) - f(b)) / (2 * h)
    return g


# central differences with h = 1e-6 in float64: h^2 truncation and 1e-16 / h rounding, both near 1e-10
TOL = 1e-7


def test_layernorm_grad_is_the_formula_s_slope():
    r = np.random.default_rng(0)
    x, dy, w, b = r.standard_normal((3, 7)), r.standard_normal((3, 7)), r.standard_normal(7), r.standard_normal(7)
    f = lambda x, w, b: (T.layernorm(x, w, b)[0] * dy).sum()  # noqa: E731
    _, mean, rstd = T.layernorm(x, w, b)
    dx, dw, db = T.layernorm_grad(dy, x, mean, rstd, w)
    assert np.allclose(dx, central(lambda v: f(v, w, b), x), rtol=0, atol=TOL)
    assert np.allclose(dw, central(lambda v: f(x, v, b), w), rtol=0, atol=TOL)
    assert np.allclose(db, central(lambda v: f(x, w, v), b), rtol=0, atol=TOL)


@pytest.mark.parametrize("renorm", [False, True])
def test_route_grad_is_the_formula_s_slope(renorm):
    r = np.random.default_rng(1)
    x, dw, topk = r.standard_normal((5, 6)), r.standard_normal((5, 2)), 2
    x[3] = -np.inf
    x[4, :5] = -np.inf
    idx, _, counts, _, _, _ = T.route(x, topk, 0.3, renorm)

    def f(v):  # the choice and the counts stay fixed: h moves no logit past another
        _, w, _, _, _, loss = T.route(v, topk, 0.3, renorm)
        return 0.7 * loss + (w * dw).sum()
    g = T.route_grad(x, idx, counts, topk, dw, 0.7, 0.3, renorm)
    live = np.isfinite(x)
    num = np.zeros_like(x)
    for i in zip(*np.nonzero(live)):
        a, b = x.copy(), x.copy()
        a[i] += 1e-6
        b[i] -= 1e-6
        num[i] = (f(a) - f(b)) / 2e-6
    assert np.allclose(g, num, rtol=0, atol=TOL)


def test_checkpoint_grid_and_scales():
    v = T.code_values()
    assert v[0x7E] == 448 and v[0x38] == 1 and v[1] == 2.0 ** -9 and np.isnan(v[0x7F]) and v[0xB8] == -1
    x = np.zeros((6, 130))
    x[0, 0], x[1, 0], x[2, 0], x[3, 0] = 448, 449, 1.75, 1.76
    x[4, :2] = [np.inf, 3.0]
    x[5, 129] = 2.0 ** -140
    unit, b = T.checkpoint(x)
    assert list(b[:, 0] - 127) == [0, 1, -8, -7, -7, -127]
    assert b[5, 1] == 0 and b[0, 1] == 0
    assert unit[0, 0] == 448 and unit[2, 0] == 448 and np.isnan(unit[4, 0]) and unit[4, 1] == 384
    r = np.random.default_rng(2).standard_normal((4, 300))
    back = T.values(*T.checkpoint(r))
    # half a step of three fraction bits; below 2^-6 of the scale's unit the step stays 2^-9
    scale = np.repeat(2.0 ** (T.checkpoint(r)[1] - 127.0), 128, 1)[:, :300]
    assert np.all(np.abs(back - r) <= np.maximum(np.abs(r) * 2.0 ** -4, scale * 2.0 ** -10))


def test_route_lists():
    x = np.array([[1.0, 3, 3, 2], [-np.inf] * 4, [-np.inf, 5, -np.inf, -np.inf], [0, 0, 0, 0]])
    idx, w, counts, offs, rows, _ = T.route(x, 2, renormalize=True)
    assert idx.tolist() == [[1, 2], [-1, -1], [1, -1], [0, 1]]
    assert counts.tolist() == [1, 3, 1, 0, 3] and offs.tolist() == [0, 1, 4, 5, 5]
    assert rows.tolist() == [6, 0, 4, 7, 1, -1, -1, -1]
    assert np.allclose(w, [[0.5, 0.5], [0, 0], [1, 0], [0.5, 0.5]])


def test_weight_grad_groups():
    r = np.random.default_rng(3)
    dy, x = r.standard_normal((6, 2)), r.standard_normal((3, 4))
    rows = np.array([0, 3, 5, 1, 2, 4])
    out, _ = T.weight_grad(dy, x, [0, 2, 2, 6], rows, 2)
    want = np.zeros((3, 2, 4))
    for g, (lo, hi) in enumerate([(0, 2), (2, 2), (2, 6)]):
        for s in range(lo, hi):
            want[g] += np.outer(dy[s], x[rows[s] // 2])
    assert np.allclose(out, want, rtol=0, atol=1e-14)
