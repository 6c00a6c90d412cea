"""Products that stream from tile to tile in 256 x 256 tiles, or take those tiles
through registers, and how exact a long sum has to be: shared by the tests on the
CPU (that the plan takes these forms, that the bounds see lost precision) and on
the GPU."""
U = 2.0 ** -24
FORWARD, GATED, BACKWARD, BOTH = range(4)  # BOTH: the gated block's dx, a sum over both products

# kind, slots, groups, columns, length of the sum, type, whether rows lie in whole 16-byte chunks (else the tiles go through
# registers). More tiles than CUs in each, so that a workgroup goes from one to the next; sums that end inside a step (64
# values of bf16, 32 of float32) and inside a chunk, of one step and a part and of several; one group without lists, and
# uneven groups.
STREAMING = [
    (kind, slots, groups, n // 2 if kind == GATED else n, k, "bf16", aligned)
    for kind in range(4) for slots, groups, n, k, aligned in (
        (20000, 1, 1032, 136, True), (8192, 1, 4096, 520, True), (20000, 24, 1032, 264, True), (20000, 40, 1032, 136, True),
        (20000, 1, 1031, 517, False), (20000, 24, 1031, 199, False), (20000, 40, 1031, 131, False))
] + [
    (kind, slots, groups, n // 2 if kind == GATED and groups > 1 else n, k, "f32", aligned)
    for kind in range(4) for slots, groups, n, k, aligned in (
        (20000, 1, 4096, 264, True), (20000, 24, 1032, 136, True), (20000, 40, 1032, 72, True), (20000, 40, 1031, 67, False))
]


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
