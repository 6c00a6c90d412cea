"""Calls of the feed-forward operators at the edge of what their documentation
allows, without a GPU: what is accepted writes nothing, what is refused is
refused on the host (addresses here are fake and never dereferenced)."""
import pytest
import torch

import muon_newton_schulz_03_amd as mu


@pytest.mark.parametrize("call", [mu.muon_expert_forward, mu.muon_expert_backward])
def test_gather_and_scatter_without_rows(call):
    """The slots are then counted by no operand: neither x nor y has a row for each."""
    t, w = torch.zeros(4, 8), torch.zeros(2, 8, 8)
    with pytest.raises(ValueError, match="rows: needed"):
        call(t, w, t, torch.zeros(3, dtype=torch.int32), gather=1, scatter=True)
