"""Refusals of the training operators, without a GPU: every invalid call is
rejected on the host with the documented status before anything is launched
(addresses here are fake and never dereferenced), the workspace sizes, and
the binding's checks of tensors."""
import ctypes
import random
import time

import pytest
import torch

import muon_newton_schulz_03_amd as mu

A = 1 << 32
BF, F32 = mu.MUON_BF16, mu.MUON_F32
INV, SHAPE, DTYPE, ALIGN, ALIAS, WORK = (mu.MUON_ERR_INVALID_ARG, mu.MUON_ERR_SHAPE, mu.MUON_ERR_DTYPE, mu.MUON_ERR_ALIGN,
                                         mu.MUON_ERR_ALIAS, mu.MUON_ERR_WORKSPACE)


def m(at, rows=4, cols=8, dtype=BF, ld=None):
    return mu.muon_mat(A * at, rows, cols, cols if ld is None else ld, dtype, 1)


def ck(at, rows=4, cols=8, ld_c=None, ld_s=None):
    groups = -(-cols // 128)
    return mu.muon_ckpt(A * at, A * at + (1 << 31), rows, cols, cols if ld_c is None else ld_c, groups if ld_s is None else ld_s)


def ref(x):
    return ctypes.byref(x) if isinstance(x, ctypes.Structure) else x


@pytest.fixture(autouse=True)
def no_workspace():
    mu.muon_set_workspace(None, 0)
    yield
    mu.muon_set_workspace(None, 0)


def call(name, *args):
    return getattr(mu.lib(), name)(*[ref(a) for a in args])


def fwd(x=m(1), y=m(2), mean=A * 3, rstd=A * 4, w=m(5, 1), b=m(6, 1), eps=1e-5, c=None):
    return call("muon_layernorm_forward", x, y, mean, rstd, w, b, eps, c)


def test_layernorm_forward_refusals():
    assert fwd(x=None) == INV and "x" in mu.muon_last_error()
    assert fwd(y=None) == INV
    assert fwd(x=m(1, dtype=7)) == DTYPE
    assert fwd(y=m(2, dtype=F32)) == DTYPE
    assert fwd(y=m(2, cols=9)) == SHAPE
    assert fwd(x=m(1, rows=-1), y=m(2, rows=-1)) == SHAPE
    assert fwd(x=m(1, cols=0), y=m(2, cols=0)) == SHAPE
    assert fwd(x=m(1, cols=32769), y=m(2, cols=32769), w=None, b=None) == SHAPE
    assert fwd(x=m(1, ld=7)) == SHAPE
    assert fwd(w=m(5, 2)) == SHAPE
    assert fwd(b=m(6, 1, 9)) == SHAPE
    assert fwd(b=m(6, 1, dtype=F32)) == DTYPE
    assert fwd(eps=-1.0) == INV and fwd(eps=float("nan")) == INV and fwd(eps=float("inf")) == INV
    assert fwd(x=mu.muon_mat(None, 4, 8, 8, BF, 1)) == INV
    assert fwd(x=mu.muon_mat(A + 1, 4, 8, 8, BF, 1)) == ALIGN
    assert fwd(mean=A * 3 + 2) == ALIGN
    assert fwd(y=m(1)) == ALIAS
    assert fwd(mean=A * 2 + 4) == ALIAS
    assert fwd(rstd=A * 3 + 12) == ALIAS
    assert fwd(c=ck(7, rows=5)) == SHAPE
    assert fwd(c=ck(7, ld_c=7)) == SHAPE
    assert fwd(c=ck(7, ld_s=0)) == SHAPE
    assert fwd(c=ck(2)) == ALIAS
    assert fwd(c=mu.muon_ckpt(None, None, 4, 8, 8, 1)) == INV
    # no rows: nothing to launch
    none = mu.muon_mat(None, 0, 8, 8, BF, 1)
    assert fwd(x=none, y=none, mean=None, rstd=None) == mu.MUON_OK


def bwd(dy=m(1), x=m(2), mean=A * 3, rstd=A * 4, dx=m(5), w=m(6, 1), dw=m(7, 1), db=m(8, 1)):
    return call("muon_layernorm_backward", dy, x, mean, rstd, dx, w, dw, db)


def test_layernorm_backward_refusals():
    assert bwd() == WORK and "workspace" in mu.muon_last_error()
    assert bwd(mean=None) == INV and bwd(rstd=None) == INV
    assert bwd(x=m(2, rows=5)) == SHAPE
    assert bwd(dx=m(5, dtype=F32)) == DTYPE
    assert bwd(dw=m(7, 1, dtype=F32)) == DTYPE
    assert bwd(db=m(8, 4)) == SHAPE
    assert bwd(dx=m(1), dw=None, db=None) == ALIAS
    assert bwd(dx=m(2), dw=None, db=None) == ALIAS
    assert bwd(rstd=A * 5, dw=None, db=None) == ALIAS
    size = mu.muon_layernorm_workspace_size(4, 8)
    mu.muon_set_workspace(A * 9, size - 4)
    assert bwd() == WORK
    mu.muon_set_workspace(A * 2, size)
    assert bwd() == ALIAS and "workspace" in mu.muon_last_error()


def test_checkpoint_refusals():
    save = lambda x=m(1), c=ck(2): call("muon_ckpt_save", x, c)  # noqa: E731
    load = lambda c=ck(2), x=m(1): call("muon_ckpt_load", c, x)  # noqa: E731
    for f, kw in ((save, {}), (load, {})):
        assert f(x=None) == INV and f(c=None) == INV
        assert f(x=m(1, cols=9)) == SHAPE and f(x=m(1, rows=3)) == SHAPE
        assert f(x=m(1, dtype=2)) == DTYPE
        assert f(x=mu.muon_mat(A + 1, 4, 8, 8, BF, 1)) == ALIGN
        assert f(c=ck(1)) == ALIAS
        assert f(c=ck(2, ld_c=3)) == SHAPE
        assert f(c=mu.muon_ckpt(A, A * 3, 4, 8, 8, 1), x=m(3)) == ALIAS
        none = mu.muon_mat(None, 0, 8, 8, BF, 1)
        assert f(x=none, c=mu.muon_ckpt(None, None, 0, 8, 8, 1)) == mu.MUON_OK
    # codes that lie between the rows of a wide matrix do not overlap it
    wide = m(1, rows=3, cols=8, ld=64)
    inside = mu.muon_ckpt(A + 16, A * 3, 3, 8, 128, 1)
    assert call("muon_ckpt_save", wide, mu.muon_ckpt(A + 15, A * 3, 3, 8, 128, 1)) == ALIAS
    assert call("muon_ckpt_save", wide, mu.muon_ckpt(A + 121, A * 3, 3, 8, 128, 1)) == ALIAS
    del inside


def wgrad(dy=m(1, 12, 6), x=ck(2, 4, 8), g=m(3, 6, 8), stride=48, groups=2, offs=A * 4, rows=A * 5, per=3):
    return call("muon_ckpt_weight_grad", dy, x, g, stride, groups, offs, rows, per)


def test_weight_grad_refusals():
    assert wgrad(dy=None) == INV and wgrad(x=None) == INV and wgrad(g=None) == INV
    assert wgrad(g=m(3, 6, 8, F32)) == DTYPE
    assert wgrad(g=m(3, 7, 8)) == SHAPE and wgrad(g=m(3, 6, 9)) == SHAPE
    assert wgrad(stride=47) == SHAPE
    assert wgrad(groups=-1) == INV and wgrad(groups=65537) == INV
    assert wgrad(offs=None) == INV
    assert wgrad(per=0) == INV
    assert wgrad(rows=None, per=2) == SHAPE
    assert wgrad(offs=A * 4 + 2) == ALIGN and wgrad(rows=A * 5 + 1) == ALIGN
    assert wgrad(g=m(1, 6, 8)) == ALIAS and wgrad(g=m(2, 6, 8)) == ALIAS
    assert wgrad(offs=A * 3 + 48 * 2) == ALIAS and wgrad(rows=A * 3) == ALIAS
    assert wgrad(groups=0, stride=0) == mu.MUON_OK
    assert call("muon_ckpt_weight_grad", m(1, 4096, 64), ck(2, 4096, 64), m(3, 64, 64), 0, 1, None, None, 1) == WORK
    assert mu.muon_ckpt_weight_grad_workspace_size(BF, 4096, 64, 64) > 0
    assert mu.muon_ckpt_weight_grad_workspace_size(BF, 64, 64, 64) == 0
    with pytest.raises(mu.MuonError):
        mu.muon_ckpt_weight_grad_workspace_size(5, 1, 1, 1)
    with pytest.raises(mu.MuonError):
        mu.muon_ckpt_weight_grad_workspace_size(BF, 1, 1 << 29, 1 << 29)


def route(x=m(1, 6, 8, F32), topk=2, renorm=1, alpha=0.1, idx=A * 2, w=A * 3, c=A * 4, o=A * 5, r=A * 6, loss=A * 7):
    return call("muon_route_forward", x, topk, renorm, alpha, idx, w, c, o, r, loss)


def test_route_refusals():
    assert route(x=None) == INV
    assert route(topk=0) == INV and route(topk=9) == INV and route(x=m(1, 6, 64, F32), topk=33) == INV
    assert route(x=m(1, 6, 1025, F32)) == SHAPE
    assert route(x=m(1, (1 << 31) - 1, 8, F32)) == SHAPE
    assert route(renorm=2) == INV and route(alpha=float("nan")) == INV
    for name in ("idx", "w", "c", "o", "r", "loss"):
        assert route(**{name: None}) == INV
        assert route(**{name: A * 9 + 2}) == ALIGN
        assert route(**{name: A}) == ALIAS
    assert route(w=A * 2 + 44) == ALIAS
    big = m(1, 1000, 8, F32)
    assert mu.muon_route_workspace_size(6, 8, 2) == 0 and mu.muon_route_workspace_size(1000, 8, 2) > 0
    assert route(x=big) == WORK


def rback(x=m(1, 6, 8, F32), topk=2, renorm=1, alpha=0.1, idx=A * 2, c=A * 3, dw=A * 4, dl=A * 5, out=m(6, 6, 8, F32)):
    return call("muon_route_backward", x, topk, renorm, alpha, idx, c, dw, dl, out)


def test_route_backward_refusals():
    assert rback(x=None) == INV and rback(out=None) == INV
    assert rback(out=m(6, 6, 9, F32)) == SHAPE and rback(out=m(6, 6, 8, BF)) == DTYPE
    assert rback(idx=None) == INV and rback(c=None) == INV
    assert rback(topk=9) == INV and rback(renorm=-1) == INV and rback(alpha=float("inf")) == INV
    assert rback(dw=A * 4 + 1) == ALIGN and rback(dl=A * 5 + 3) == ALIGN
    assert rback(out=m(1, 6, 8, F32)) == ALIAS and rback(dw=A * 6) == ALIAS
    none = mu.muon_mat(None, 0, 8, 8, F32, 1)
    assert rback(x=none, out=none, idx=None, c=None, dw=None, dl=None) == mu.MUON_OK


def test_binding_refuses_what_no_kernel_may_touch():
    t = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="GPU tensor"):
        mu.muon_layernorm_forward(t, t.clone())
    with pytest.raises(ValueError, match="GPU tensor"):
        mu.muon_route_backward(t, t, t, t)
    codes, scales = torch.zeros((4, 8), dtype=torch.float8_e4m3fn), torch.zeros((4, 1), dtype=torch.uint8)
    with pytest.raises(ValueError, match="GPU tensor"):
        mu.Checkpoint(codes, scales)
    with pytest.raises(TypeError):
        mu.Checkpoint(t, scales)
    with pytest.raises(ValueError, match="scales"):
        mu.Checkpoint(codes, scales[:3])


def test_exchanging_the_workspace():
    p, n = ctypes.c_void_p(), ctypes.c_size_t()
    swap = mu.lib().muon_exchange_workspace
    assert swap(A, 512, p, n) == mu.MUON_OK and not p.value and n.value == 0
    assert swap(A * 2 + 1, 256, p, n) == ALIGN and swap(None, 256, p, n) == INV
    assert not p.value and n.value == 0
    assert swap(A * 2, 256, p, n) == mu.MUON_OK and p.value == A and n.value == 512
    assert swap(p, n, None, None) == mu.MUON_OK
    assert mu.lib().muon_get_workspace(p, n) == mu.MUON_OK and p.value == A and n.value == 512


def test_pitches_whose_offsets_pass_64_bits():
    far = 1 << 61
    assert fwd(x=m(1, ld=far)) == SHAPE and fwd(y=m(2, ld=far)) == SHAPE
    assert fwd(c=ck(7, ld_c=far)) == SHAPE and fwd(c=ck(7, ld_s=far)) == SHAPE
    assert wgrad(g=m(3, 6, 8, ld=far)) == SHAPE and wgrad(stride=far) == SHAPE
    assert rback(out=m(6, 6, 8, F32, ld=far)) == SHAPE


MOST = (1 << 31) - (1 << 22)  # slots, and with them tokens, that 32-bit counters can step past


@pytest.mark.parametrize("topk", [1, 2, 8])
def test_routing_counts_that_device_counters_cannot_pass(topk):
    most = MOST // topk
    assert mu.muon_route_workspace_size(most, 8, topk) > 0
    for tokens in (most + 1, ((1 << 31) - 1) // topk):
        with pytest.raises(mu.MuonError) as e:
            mu.muon_route_workspace_size(tokens, 8, topk)
        assert e.value.status == SHAPE
        x = m(1, tokens, 8)
        assert route(x=x, topk=topk, idx=A * 64, w=A * 96, c=A * 128, o=A * 160, r=A * 192, loss=A * 224) == SHAPE
        assert rback(x=x, topk=topk, idx=A * 64, c=A * 128, dw=A * 160, dl=A * 192, out=m(256, tokens, 8)) == SHAPE


def test_weight_grad_slots_that_device_counters_cannot_pass():
    size = mu.muon_ckpt_weight_grad_workspace_size
    assert size(BF, MOST, 8, 8, 1) > 0 and size(F32, MOST, 4096, 4096, 1) == 0
    for slots in (MOST + 1, (1 << 31) - 1):
        for dtype in (BF, F32):
            with pytest.raises(mu.MuonError) as e:
                size(dtype, slots, 8, 8, 1)
            assert e.value.status == SHAPE
            assert wgrad(dy=m(1, slots, 8, dtype), x=ck(64, 1, 8), g=m(65, 8, 8, dtype), groups=1, offs=None, rows=A * 66,
                         per=1) == SHAPE


def test_checkpoint_tensors_are_its_own(monkeypatch):
    """A call takes the memory that the checkpoint's tensors have then, and never memory that is gone (the
    descriptor stands for a call here; every tensor says that it is on a GPU)."""
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 0)
    new = lambda rows=4, cols=200: torch.zeros((rows, cols), dtype=torch.float8_e4m3fn)  # noqa: E731
    codes, scales = new(), torch.zeros((4, 2), dtype=torch.uint8)
    c = mu.Checkpoint(codes, scales)
    at = lambda: mu.muon_ckpt.from_buffer_copy(c._desc(0))  # noqa: E731
    assert (at().codes, at().scales, at().rows, at().cols) == (codes.data_ptr(), scales.data_ptr(), 4, 200)
    with pytest.raises(AttributeError):
        c.codes = new()
    with pytest.raises(AttributeError):
        c.scales = scales.clone()
    assert c.codes is codes and c.scales is scales and c.shape == (4, 200)
    old, other = codes.data, new()
    codes.data = other
    assert at().codes == other.data_ptr() != old.data_ptr()
    codes.data = new(4, 384)[:, :200]
    assert at().ld_codes == 384
    codes.data = new(3)
    with pytest.raises(ValueError, match="scales"):
        at()
    codes.data = new(5)[1:]
    assert at().codes == codes.data_ptr()
    codes.untyped_storage().resize_(0)
    with pytest.raises(ValueError, match="freed"):
        at()
    scales.untyped_storage().resize_(0)
    with pytest.raises(ValueError, match="freed"):
        at()


def x_meets_y(x, y):
    """Whether the overlap check finds x and y to share a byte: the statistics overlap too, so that every call is refused."""
    assert fwd(x=x, y=y, mean=A * 80, rstd=A * 80, w=None, b=None) == ALIAS
    text = mu.muon_last_error()
    assert text in ("x and y overlap", "mean and rstd overlap")
    return text == "x and y overlap"


def test_overlap_check_against_every_byte():
    r = random.Random(0)
    seen = [0, 0]
    for _ in range(4000):
        rows, cols = r.randint(1, 6), r.randint(1, 9)
        ld = [cols + r.randint(0, 14) for _ in range(2)]
        if r.random() < 0.6:
            ld[1] = ld[0]
        at = 2 * r.randint(-60, 60)
        x, y = m(40, rows, cols, ld=ld[0]), mu.muon_mat(A * 40 + at, rows, cols, ld[1], BF, 1)
        mine = {2 * (i * ld[0] + j) + b for i in range(rows) for j in range(cols) for b in range(2)}
        other = {at + 2 * (i * ld[1] + j) + b for i in range(rows) for j in range(cols) for b in range(2)}
        shared = not mine.isdisjoint(other)
        assert x_meets_y(x, y) == shared, (rows, cols, ld, at)
        seen[shared] += 1
    assert min(seen) > 500


def test_overlap_check_of_many_interleaved_rows():
    """Two halves of a wide buffer, 2^30 rows: found apart (or a byte into each other) without a walk over the rows."""
    start = time.perf_counter()
    x = m(40, 1 << 30, 4, ld=8)
    assert not x_meets_y(x, mu.muon_mat(A * 40 + 8, 1 << 30, 4, 8, BF, 1))
    assert x_meets_y(x, mu.muon_mat(A * 40 + 6, 1 << 30, 4, 8, BF, 1))
    # the last row of x under the first of y
    far = ((1 << 30) - 1) * 16
    assert x_meets_y(x, mu.muon_mat(A * 40 + far, 1 << 30, 4, 8, BF, 1))
    assert not x_meets_y(x, mu.muon_mat(A * 40 + far + 8, 1 << 30, 4, 8, BF, 1))
    assert time.perf_counter() - start < 0.5
