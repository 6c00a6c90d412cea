"""Long sums that workgroups share, against 64-bit sums on the GPU in norm, where
lost precision shows."""
import pytest
import torch

from ff_forms import tight
from test_gpu_ff_ops import BF, F32, LONG, gen, grouped64, mat, out_mat, stack

pytestmark = pytest.mark.gpu


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
