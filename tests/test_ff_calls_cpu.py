"""Calls of the feed-forward operators at the edge of what their documentation
allows, without a GPU: what is accepted writes nothing, what is refused is
refused on the host (addresses here are fake and never dereferenced)."""
import ctypes

import pytest
import torch

import muon_newton_schulz_03_amd as mu


@pytest.mark.parametrize("call", [mu.muon_expert_forward, mu.muon_expert_backward])
def test_gather_and_scatter_without_rows(call):
    """The slots are then counted by no operand: neither x nor y has a row for each."""
    t, w = torch.zeros(4, 8), torch.zeros(2, 8, 8)
    with pytest.raises(ValueError, match="rows: needed"):
        call(t, w, t, torch.zeros(3, dtype=torch.int32), gather=1, scatter=True)


A = 1 << 36
BF, F32 = mu.MUON_BF16, mu.MUON_F32


def m(at, rows, cols, dtype=BF):
    return mu.muon_mat(A * at if at else None, rows, cols, cols, dtype, 1)


def call(name, *args):
    return getattr(mu.lib(), name)(*[ctypes.byref(a) if isinstance(a, ctypes.Structure) else a for a in args])


def test_weights_of_no_groups_have_no_data():
    """A rank without experts: an empty stack's address is NULL. With a group it is refused."""
    def calls(groups):
        x, h, g = m(1, 12, 8), m(2, 12, 6), [m(i, 12, 6) for i in (3, 4, 5, 6)]
        w, wt = m(0, 6, 8), m(0, 8, 6)
        ckpt = mu.muon_ckpt(A * 7, A * 8, 12, 8, 8, 1)
        return [call("muon_gated_forward", x, w, 48, w, 48, groups, A * 9, A * 10, 1, 0, h, None, None),
                call("muon_gated_backward", h, g[0], g[1], w, 48, w, 48, groups, A * 9, A * 10, 0, g[2], g[3], x),
                call("muon_expert_forward", x, w, 48, groups, 12, A * 9, None, 0, 0, h),
                call("muon_expert_backward", x, wt, 48, groups, 12, A * 9, None, 0, 0, h),
                call("muon_ckpt_weight_grad", h, ckpt, w, 48, groups, A * 9, None, 1)]
    assert calls(0) == [mu.MUON_OK] * 5
    assert calls(1) == calls(2) == [mu.MUON_ERR_INVALID_ARG] * 5


def test_no_slots_leave_dx_of_any_rows():
    """A rank that no token came to: rows of no slots have no address, and dx, whose rows they would name, its own number of
    rows; nothing is written."""
    w = m(1, 6, 8)
    back = lambda slots, dx: call("muon_gated_backward", *(m(i if slots else 0, slots, 6) for i in (2, 3, 4)), w, 48, w, 48, 2, A * 5,  # noqa: E731
                                  None, 0, *(m(i if slots else 0, slots, 6) for i in (6, 7)), dx)
    assert back(0, m(8, 15, 8)) == back(0, m(0, 0, 8)) == mu.MUON_OK
    assert back(12, m(8, 15, 8)) == mu.MUON_ERR_SHAPE
