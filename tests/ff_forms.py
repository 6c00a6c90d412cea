"""How exact a long sum has to be: shared by the tests on the CPU (that the bound
sees lost precision) and on the GPU."""
U = 2.0 ** -24


def tight(got, ref, terms, what):
    """The norm of the error of float32 sums of `terms` independent terms, rounded once to got's type.

    Each of at most `terms` additions is off by at most 2 u of what has been added so far (a matrix instruction may cut, half a
    step twice over), which after i of them has sqrt(i / terms) of the sum's norm: 4/3 terms u by the triangle inequality. A
    float32 product adds at most u of itself. The last rounding's error is that of the exact values' in norm, and at right
    angles to the sum's error, but for where values happen to fall: over n normal values the norm of both spreads by
    1 / sqrt(n), and four times that is allowed."""
    ref = ref.double()
    rounding, sums = float((ref.to(got.dtype).double() - ref).norm()), (4 * terms / 3 + 2) * U * float(ref.norm())
    bound = (rounding ** 2 + sums ** 2) ** 0.5 * (1 + 4 * ref.numel() ** -0.5)
    off = float((got.double() - ref).norm())
    assert off <= bound, f"{what}: the error's norm is {off / max(bound, 1e-300):.3g} of what it may be"
