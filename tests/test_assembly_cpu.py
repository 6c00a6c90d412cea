"""Inline assembly in the kernels' sources tells the compiler what it writes."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "muon_newton_schulz_03_amd", "csrc")
SOURCES = sorted(f for f in os.listdir(CSRC) if f.endswith((".hip", ".h")))


def statements(text):
    """The arguments of each asm statement: what stands between its parentheses."""
    for m in re.finditer(r"\basm\s+volatile\s*\(", text):
        depth, at = 1, m.end()
        while depth:
            depth += {"(": 1, ")": -1}.get(text[at], 0)
            at += 1
        yield text[m.end():at - 1]


@pytest.mark.parametrize("source", SOURCES)
def test_scalar_registers_that_assembly_writes_are_clobbers(source):
    with open(os.path.join(CSRC, source)) as f:
        text = f.read()
    for body in statements(text):
        code = body.split("\"\n")[0]
        for register in re.findall(r"\bs_mov_b32 (m0|vcc\w*|s\d+)\b", code):
            assert f'"{register}"' in body, f"{source}: {register} is written and not named: {body!r}"
