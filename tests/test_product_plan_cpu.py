"""Which tiles the products take (product_plan.cpp, which runs on the host), built
with g++ under AddressSanitizer and UndefinedBehaviorSanitizer: the sizes of the
GPU tests take the forms that those tests are for, and every product kernel of the
library is one that some call takes."""
import os
import re
import shutil
import subprocess

import pytest

import muon_newton_schulz_03_amd as mu
from ff_forms import BACKWARD, BOTH, FORWARD, GATED, STREAMING

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "muon_newton_schulz_03_amd", "csrc")
LARGE, WIDE, SMALL, MID, THIN, THIN2 = range(6)


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("g++ not installed")
    exe = tmp_path_factory.mktemp("plan") / "product_plan_test"
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-D__HIP_PLATFORM_AMD__",
           "-I/opt/rocm/include", "-I", CSRC, os.path.join(ROOT, "tests", "product_plan_test.cpp"),
           os.path.join(CSRC, "product_plan.cpp"), "-o", str(exe)]
    build = subprocess.run(cmd, capture_output=True, text=True)
    assert build.returncode == 0, build.stdout + build.stderr

    def ask(args, lines):
        run = subprocess.run([str(exe), *args], input="\n".join(" ".join(map(str, line)) for line in lines), capture_output=True,
                             text=True, timeout=300)
        assert run.returncode == 0 and not run.stderr, run.stdout + run.stderr
        return [tuple(map(int, line.split())) for line in run.stdout.splitlines()]
    return ask


def test_streaming_sizes_stream(plan):
    """256 x 256 tiles, nothing shared out, more of them than CUs: every kind, with one group and with several."""
    asked = [(int(dtype == "bf16"), kind, int(aligned), slots, groups, n, k) for kind, slots, groups, n, k, dtype, aligned in STREAMING]
    for size, got in zip(asked, plan([], asked)):
        _, kind, _, slots, groups, n, _ = size
        assert got == (LARGE, 0, 0, 0), (size, got)
        least = -(-slots // 256) if groups == 1 else slots // 256  # row tiles, however the slots fall
        assert least * -(-n // (128 if kind == GATED else 256)) > 256, size
    for kind in (FORWARD, GATED, BACKWARD, BOTH):
        for bf16 in (0, 1):
            for lds in (0, 1):
                assert any(a[:3] == (bf16, kind, lds) for a in asked), (bf16, kind, lds)


def test_forms_of_the_sizes_named_in_comments(plan):
    """The sizes beside the estimate, with the form that each is said to take."""
    sizes = {(1, GATED, 1, 8, 128, 768, 2048): THIN, (1, GATED, 1, 640, 89, 418, 135): WIDE, (1, FORWARD, 1, 1024, 1, 2048, 2048): SMALL,
             (1, FORWARD, 1, 2048, 1, 4096, 4096): WIDE, (1, GATED, 1, 32768, 128, 768, 2048): LARGE,
             (1, FORWARD, 0, 8192, 1, 4095, 2047): LARGE, (0, FORWARD, 1, 1024, 1, 1024, 2048): THIN2,
             (0, GATED, 1, 2331, 12, 532, 1024): MID, (0, FORWARD, 1, 4096, 1, 2048, 4096): SMALL}
    got = plan([], sizes)
    assert {size: g[0] for size, g in zip(sizes, got) if g[2] == 0} == sizes


def test_every_kernel_is_reached(plan):
    """The product kernels that the library was compiled with are those that some size takes."""
    if shutil.which("nm") is None:
        pytest.skip("nm not installed")
    names = subprocess.run(["nm", mu.LIB_PATH], capture_output=True, text=True, check=True).stdout
    forms = {(2, 4, 4, 1, 128, 1): LARGE, (2, 4, 4, 1, 128, 0): LARGE, (1, 4, 4, 1, 64, 0): WIDE, (2, 2, 1, 1, 128, 0): SMALL,
             (2, 1, 1, 2, 64, 0): MID, (1, 1, 1, 4, 128, 0): THIN, (1, 1, 1, 4, 64, 0): THIN2}
    built = set()
    for t, wm, wn, i, kk, _, row, stream, back, gated, direct, part in re.findall(
            r"stub__product_kernelI(DF16b|f)NS0_4FormILi(\d)ELi(\d)ELi(\d)ELi(\d)ELi(\d)ELi(\d+)ELb(\d)EEELb(\d)ELb(\d)ELb(\d)ELb(\d)E", names):
        form = forms[tuple(map(int, (wm, wn, i, kk, row, stream)))]
        built.add((int(t != "f"), 2 if back == "1" else int(gated), int(direct), form, int(part)))
    assert built
    assert built == set(plan(["all"], []))
