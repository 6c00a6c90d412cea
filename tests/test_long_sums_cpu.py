"""How exact the GPU tests hold long sums to be."""
import pytest
import torch

from ff_forms import U, tight


@pytest.mark.parametrize("terms", [700, 4095, 12288])
def test_the_bound_of_long_sums_sees_lost_precision(terms):
    """Float32 sums of 16 parts pass; parts or operands in bf16, or a sum that lacks its last term, do not."""
    g = torch.Generator().manual_seed(terms)
    x, w = torch.randn((48, terms), generator=g), torch.randn((64, terms), generator=g) * terms ** -0.5
    ref = x.double() @ w.double().t()

    def parts(x, w, keep=lambda p: p):
        return sum(keep(a @ b.t()) for a, b in zip(x.split(-(-terms // 16), 1), w.split(-(-terms // 16), 1)))

    bf = lambda t: t.to(torch.bfloat16).float()  # noqa: E731
    tight(parts(x, w), ref, terms, "float32")
    tight(parts(x, w).to(torch.bfloat16), ref, terms, "float32, rounded to bf16")
    for wrong in (parts(x, w, bf), parts(bf(x), bf(w)), parts(x[:, :-1], w[:, :-1])):
        with pytest.raises(AssertionError):
            tight(wrong, ref, terms, "wrong")
        with pytest.raises(AssertionError):
            tight(wrong.to(torch.bfloat16), ref, terms, "wrong, rounded to bf16")
    assert (4 * terms / 3 + 2) * U < 1e-3
