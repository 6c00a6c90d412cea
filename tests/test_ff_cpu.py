"""Refusals of the feed-forward operators, without a GPU: every invalid call is
rejected on the host with the documented status before anything is launched
(addresses here are fake and never dereferenced), and the binding's checks; the
oracles against closed forms and differences."""
import ctypes

import numpy as np
import pytest
import torch

import muon_newton_schulz_03_amd as mu
from oracle import ff_oracle as F

A = 1 << 36
BF, F32 = mu.MUON_BF16, mu.MUON_F32
INV, SHAPE, DTYPE, ALIGN, ALIAS, WORK = (mu.MUON_ERR_INVALID_ARG, mu.MUON_ERR_SHAPE, mu.MUON_ERR_DTYPE, mu.MUON_ERR_ALIGN,
                                         mu.MUON_ERR_ALIAS, mu.MUON_ERR_WORKSPACE)
MOST = (1 << 31) - (1 << 22)


def m(at, rows=4, cols=8, dtype=BF, ld=None):
    return mu.muon_mat(A * at, rows, cols, cols if ld is None else ld, dtype, 1)


def odd(at, rows=4, cols=8):
    return mu.muon_mat(A * at + 1, rows, cols, cols, BF, 1)


def ref(x):
    return ctypes.byref(x) if isinstance(x, ctypes.Structure) else x


@pytest.fixture(autouse=True)
def no_workspace():
    mu.muon_set_workspace(None, 0)
    yield
    mu.muon_set_workspace(None, 0)


def call(name, *args):
    return getattr(mu.lib(), name)(*[ref(a) for a in args])


# 12 slots of 5 tokens (3 each at most), 2 groups, n 6, k 8

def gated(x=m(1, 5), wg=m(2, 6), gs=48, wu=m(3, 6), us=48, groups=2, offs=A * 4, rows=A * 5, per=3, act=0, h=m(6, 12, 6),
          gate=m(7, 12, 6), up=m(8, 12, 6)):
    return call("muon_gated_forward", x, wg, gs, wu, us, groups, offs, rows, per, act, h, gate, up)


def test_gated_forward_refusals():
    for name in ("x", "wg", "wu", "h"):
        assert gated(**{name: None}) == INV, name
    assert gated(x=m(1, 5, dtype=7)) == DTYPE and gated(x=m(1, 5, dtype=F32)) == DTYPE
    assert gated(wg=m(2, 6, dtype=F32)) == DTYPE and gated(wu=m(3, 6, dtype=F32)) == DTYPE
    assert gated(h=m(6, 12, 6, F32)) == DTYPE and gated(gate=m(7, 12, 6, F32)) == DTYPE and gated(up=m(8, 12, 6, F32)) == DTYPE
    assert gated(wg=m(2, 7)) == SHAPE and gated(wu=m(3, 7)) == SHAPE and gated(wg=m(2, 6, 9), wu=m(3, 6, 9)) == SHAPE
    assert gated(wg=m(2, 0), wu=m(3, 0)) == SHAPE
    assert gated(gate=m(7, 11, 6)) == SHAPE and gated(up=m(8, 12, 7)) == SHAPE and gated(x=m(1, 5, 9)) == SHAPE
    assert gated(gs=47) == SHAPE and gated(us=0) == SHAPE and gated(gs=1 << 61) == SHAPE
    assert gated(h=m(6, 12, 6, ld=5)) == SHAPE and gated(h=m(6, 12, 6, ld=1 << 61)) == SHAPE
    assert gated(groups=-1) == INV and gated(groups=65537) == INV and gated(offs=None) == INV
    assert gated(per=0) == INV and gated(act=2) == INV and gated(act=-1) == INV
    assert gated(rows=None, per=2) == SHAPE
    assert gated(offs=A * 4 + 2) == ALIGN and gated(rows=A * 5 + 1) == ALIGN and gated(x=odd(1, 5)) == ALIGN
    assert gated(h=m(1, 12, 6)) == ALIAS and gated(h=m(2, 12, 6)) == ALIAS and gated(up=m(7, 12, 6)) == ALIAS
    assert gated(gate=m(3, 12, 6)) == ALIAS and gated(offs=A * 6) == ALIAS and gated(rows=A * 8 + 4) == ALIAS
    # the second group's weights
    assert gated(h=mu.muon_mat(A * 2 + 96 + 94, 12, 6, 6, BF, 1)) == ALIAS
    for far in (MOST + 1, (1 << 31) - 1):
        assert gated(h=m(6, far, 6), gate=None, up=None) == SHAPE
    assert gated(wg=m(2, 1 << 30), wu=m(3, 1 << 30), h=m(6, 12, 1 << 30), gate=None, up=None) == SHAPE
    assert gated(groups=0, gs=0, us=0) == mu.MUON_OK
    assert gated(h=m(6, 0, 6), gate=None, up=None) == mu.MUON_OK


def gback(dh=m(1, 12, 6), gate=m(2, 12, 6), up=m(3, 12, 6), wg=m(4, 6), gs=48, wu=m(5, 6), us=48, groups=2, offs=A * 6,
          rows=A * 7, act=0, dg=m(8, 12, 6), du=m(9, 12, 6), dx=m(10, 15)):
    return call("muon_gated_backward", dh, gate, up, wg, gs, wu, us, groups, offs, rows, act, dg, du, dx)


def test_gated_backward_refusals():
    for name in ("dh", "gate", "up", "wg", "wu", "dg", "du"):
        assert gback(**{name: None}) == INV, name
    for name, at in (("gate", 2), ("up", 3), ("dg", 8), ("du", 9)):
        assert gback(**{name: m(at, 12, 6, F32)}) == DTYPE and gback(**{name: m(at, 11, 6)}) == SHAPE, name
        assert gback(**{name: odd(at, 12, 6)}) == ALIGN
    assert gback(wg=m(4, 6, dtype=F32)) == DTYPE and gback(dx=m(10, 15, dtype=F32)) == DTYPE
    assert gback(wg=m(4, 7), wu=m(5, 7)) == SHAPE and gback(dx=m(10, 15, 9)) == SHAPE
    assert gback(rows=None) == SHAPE and gback(rows=None, dx=m(10, 12), groups=0) == mu.MUON_OK
    assert gback(act=5) == INV and gback(offs=None) == INV and gback(gs=40) == SHAPE
    for a, b in (("dg", "dh"), ("dg", "gate"), ("du", "up"), ("dg", "du")):
        at = {"dh": 1, "gate": 2, "up": 3, "du": 9}[b]
        assert gback(**{a: m(at, 12, 6)}) == ALIAS
    assert gback(dx=m(8, 15)) == ALIAS and gback(dx=m(5, 15)) == ALIAS and gback(dx=m(7, 15)) == ALIAS
    assert gback(dx=None, wg=None, wu=None, groups=0) == mu.MUON_OK


def expert(name, x=m(1, 12, 8), w=m(2, 6, 8), gs=48, groups=2, slots=12, offs=A * 3, rows=A * 4, gather=0, scatter=0, y=m(5, 12, 6)):
    return call(name, x, w, gs, groups, slots, offs, rows, gather, scatter, y)


@pytest.mark.parametrize("back", [False, True])
def test_expert_refusals(back):
    def f(**kw):
        if back:
            kw.setdefault("w", m(2, 8, 6))
        return expert("muon_expert_backward" if back else "muon_expert_forward", **kw)
    for name in ("x", "w", "y"):
        assert f(**{name: None}) == INV
    assert f(y=m(5, 12, 6, F32)) == DTYPE and f(w=m(2, 8, 6, F32) if back else m(2, 6, 8, F32)) == DTYPE
    assert f(w=m(2, 6, 8) if back else m(2, 8, 6)) == SHAPE
    assert f(x=m(1, 11)) == SHAPE and f(y=m(5, 11, 6)) == SHAPE and f(slots=11) == SHAPE and f(slots=-1) == SHAPE
    assert f(slots=MOST + 1, x=m(1, MOST + 1), y=m(5, MOST + 1, 6)) == SHAPE
    assert f(gather=-1) == INV and f(scatter=2) == INV and f(rows=None, gather=1) == INV and f(rows=None, scatter=1) == INV
    assert f(offs=None) == INV and f(groups=-1) == INV and f(gs=47) == SHAPE
    assert f(offs=A * 3 + 1) == ALIGN and f(rows=A * 4 + 2) == ALIGN
    assert f(y=m(1, 12, 6)) == ALIAS and f(y=m(2, 12, 6)) == ALIAS and f(rows=A * 5) == ALIAS
    assert f(groups=0, gs=0) == mu.MUON_OK
    assert f(x=m(1, 0), y=m(5, 0, 6), slots=0) == mu.MUON_OK
    assert f(x=m(1, 3), y=m(5, 99, 6), slots=0, gather=2, scatter=1) == mu.MUON_OK


@pytest.mark.parametrize("gated_", [False, True])
def test_product_workspace(gated_):
    """Sizes, their refusals, and calls without the workspace or with one in the way."""
    f = mu.muon_gated_workspace_size if gated_ else mu.muon_expert_workspace_size
    for args in ((2, 4, 5, 6), (F32, -1, 5, 6), (F32, MOST + 1, 5, 6), (F32, 4, 0, 6), (F32, 4, 5, 0), (F32, 4, 1 << 30, 6),
                 (F32, 4, 5, 1 << 30), (F32, 4, 5, 6, -1), (F32, 4, 5, 6, 65537), (F32, 4, 5, 6, 1, 2), (F32, 4, 5, 6, 1, -1)):
        with pytest.raises(mu.MuonError):
            f(*args)
    assert f(BF, 12, 6, 8, 2) == f(F32, 0, 6, 1 << 20) == f(F32, 5, 6, 1 << 20, 0) == f(BF, 8192, 768, 2048, 128) == 0
    size = f(F32, 12, 6, 1 << 14, 2)
    assert size > 0 and size % (12 * 6 * 4) == 0 and f(F32, 12, 1 << 14, 6, 2, 1) > 0
    x, w, y = m(1, 12, 1 << 14, F32), m(2, 6, 1 << 14, F32), m(6, 12, 6, F32)
    gs = 6 << 14
    run = lambda **kw: (gated(x=x, wg=w, wu=m(3, 6, 1 << 14, F32), gs=gs, us=gs, rows=None, per=1, h=y, gate=None, up=None, **kw)  # noqa: E731
                        if gated_ else expert("muon_expert_forward", x=x, w=w, gs=gs, y=y, **kw))
    assert run() == WORK
    mu.muon_set_workspace(A * 9, size - 4)
    assert run() == WORK
    for at in (1, 2, 4, 6):
        mu.muon_set_workspace(A * at, size)
        assert run() == ALIAS, at


def comb(x=m(1, 12), topk=3, w=A * 2, idx=A * 3, res=m(4, 4), p=0.1, key=A * 5, y=m(6, 4)):
    return call("muon_combine_forward", x, topk, w, idx, res, p, key, y)


def test_combine_refusals():
    assert comb(x=None) == INV and comb(y=None) == INV and comb(key=None) == INV
    assert comb(topk=0) == INV and comb(topk=33) == INV and comb(topk=4) == SHAPE and comb(topk=2) == SHAPE
    for p in (-0.1, 1.0, 2.0, float("nan"), float("inf")):
        assert comb(p=p) == INV
    assert comb(x=m(1, 12, 9)) == SHAPE and comb(res=m(4, 5)) == SHAPE and comb(res=m(4, 4, 9)) == SHAPE
    assert comb(x=m(1, 12, dtype=F32)) == DTYPE and comb(res=m(4, 4, dtype=F32)) == DTYPE
    assert comb(w=A * 2 + 2) == ALIGN and comb(idx=A * 3 + 1) == ALIGN and comb(key=A * 5 + 4) == ALIGN
    assert comb(y=m(1, 4)) == ALIAS and comb(y=m(4, 4)) == ALIAS and comb(w=A * 6 + 8) == ALIAS and comb(idx=A * 6) == ALIAS
    assert comb(key=A * 6 + 16) == ALIAS
    none = mu.muon_mat(None, 0, 8, 8, BF, 1)
    assert comb(x=none, y=none, res=none) == mu.MUON_OK
    assert comb(x=none, y=none, res=None, p=0.0, key=None, w=None, idx=None) == mu.MUON_OK


def cback(dy=m(1, 4), x=m(2, 12), topk=3, w=A * 3, idx=A * 4, rows=A * 5, p=0.1, key=A * 6, dx=m(7, 12), dw=A * 8):
    return call("muon_combine_backward", dy, x, topk, w, idx, rows, p, key, dx, dw)


def test_combine_backward_refusals():
    assert cback() == WORK and "workspace" in mu.muon_last_error()
    size = mu.muon_combine_workspace_size(4, 3)
    assert size == 48
    mu.muon_set_workspace(A * 9, size - 4)
    assert cback() == WORK
    mu.muon_set_workspace(A * 7, size)
    assert cback() == ALIAS
    for name in ("dy", "x", "dx"):
        assert cback(rows=None, **{name: None}) == INV
    assert cback(rows=None, dx=m(7, 11)) == SHAPE and cback(rows=None, x=m(2, 11)) == SHAPE and cback(rows=None, topk=4) == SHAPE
    assert cback(rows=None, dx=m(7, 12, dtype=F32)) == DTYPE and cback(rows=None, x=m(2, 12, dtype=F32)) == DTYPE
    assert cback(rows=A * 5 + 2) == ALIGN and cback(rows=None, dw=A * 8 + 1) == ALIGN
    assert cback(rows=None, dx=m(1, 12)) == ALIAS and cback(rows=None, dx=m(2, 12)) == ALIAS and cback(rows=None, dw=A * 7) == ALIAS
    assert cback(rows=None, dw=A * 3) == ALIAS and cback(rows=None, p=1.0) == INV and cback(rows=None, key=None) == INV
    none = mu.muon_mat(None, 0, 8, 8, BF, 1)
    assert cback(dy=none, x=none, dx=none, rows=A * 5) == mu.MUON_OK
    for tokens, topk in ((-1, 1), (1 << 30, 2), (1, 0), (1, 33)):
        with pytest.raises(mu.MuonError):
            mu.muon_combine_workspace_size(tokens, topk)


def test_dropout_refusals():
    fwd = lambda x=m(1), res=m(2), p=0.1, key=A * 3, y=m(4): call("muon_dropout_forward", x, res, p, key, y)  # noqa: E731
    bwd = lambda x=m(1), p=0.1, key=A * 3, y=m(4): call("muon_dropout_backward", x, p, key, y)  # noqa: E731
    assert fwd(res=m(2, 5)) == SHAPE and fwd(y=m(2)) == ALIAS
    for f in (fwd, bwd):
        assert f(x=None) == INV and f(y=None) == INV and f(key=None) == INV and f(p=1.0) == INV
        assert f(x=m(1, 5)) == SHAPE and f(x=m(1, cols=9)) == SHAPE and f(x=m(1, dtype=F32)) == DTYPE
        assert f(y=m(1)) == ALIAS and f(key=A * 4) == ALIAS and f(key=A * 3 + 4) == ALIGN


def test_binding_refuses_what_no_kernel_may_touch():
    t, w = torch.zeros(4, 8), torch.zeros(2, 6, 8)
    for f, args in ((mu.muon_gated_forward, (t, w, w, t)), (mu.muon_gated_backward, (t, t, t, w, w, t, t, t)),
                    (mu.muon_expert_forward, (t, w, t)), (mu.muon_expert_backward, (t, w, t)),
                    (mu.muon_combine_forward, (t, t)), (mu.muon_combine_backward, (t, t, t)),
                    (mu.muon_dropout_forward, (t, t, 0.1)), (mu.muon_dropout_backward, (t, t, 0.1))):
        with pytest.raises(ValueError, match="GPU tensor"):
            f(*args)


def test_words_of_the_generator():
    """The published test vectors of Philox4x32-10 (zeros, ones, digits of pi), and blocks whose counter passes 32 bits."""
    for counter, key, words in (
            ((0, 0, 0, 0), (0, 0), (0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8)),
            ((0xffffffff,) * 4, (0xffffffff,) * 2, (0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd)),
            ((0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344), (0xa4093822, 0x299f31d0), (0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1))):
        assert tuple(int(v) for v in F.philox(counter, key)) == words
    whole = F.kept(2 ** 34 - 8, 16, 0.5, 5, -1)
    assert np.array_equal(F.kept(2 ** 34 - 3, 9, 0.5, 5, -1), whole[5:14])
    share = F.kept(0, 200000, 0.3, 1, 2).mean()
    assert abs(share - 0.7) < 5 * (0.21 / 200000) ** 0.5


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_slopes_of_activations(kind):
    g = np.linspace(-8, 8, 161)
    step = 1e-5
    difference = (F.act(g + step, kind)[0] - F.act(g - step, kind)[0]) / (2 * step)
    assert np.allclose(F.act(g, kind)[1], difference, atol=1e-9)
    t = torch.from_numpy(g)
    want = torch.nn.functional.silu(t) if kind == "silu" else torch.nn.functional.gelu(t)
    assert np.allclose(F.act(g, kind)[0], want.numpy(), atol=1e-14)


def test_product_oracle():
    r = np.random.RandomState(0)
    x, w = r.randn(5, 4), r.randn(2, 3, 4)
    y, mag, used = F.product(x, w, [1, 3, 4], 5, [0, 4, -1, 2, 1])
    assert np.allclose(y[1], w[0] @ x[4]) and not y[2].any() and np.allclose(y[3], w[1] @ x[2])
    assert list(used) == [False, True, True, True, False] and np.all(mag >= np.abs(y) - 1e-12)
    z, _, _ = F.product(r.randn(3, 3), w, None, 3, back=True)
    assert z.shape == (3, 4)
