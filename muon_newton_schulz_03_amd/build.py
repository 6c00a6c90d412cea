"""Builds libmuon.so (HIP kernels + C ABI) for gfx950, in place.

    python -m muon_newton_schulz_03_amd.build

Compiles every source under csrc/ with hipcc, several at a time. Every HIP
translation unit is built with packed-fp32 instructions disabled.
"""
import concurrent.futures
import os
import shutil
import subprocess
import sys
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libmuon.so")
ARCH = "gfx950"


def hipcc():
    for cand in (os.environ.get("HIPCC"), shutil.which("hipcc"), "/opt/rocm/bin/hipcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found")


def build(verbose=False):
    sources = sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC)
                     if f.endswith((".hip", ".cpp")))
    flags = [hipcc(), f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC",
             "-Wall", "-Wno-unused-function",
             "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
             "-I", INCLUDE, "-I", CSRC]

    def run(cmd):
        if verbose:
            print(" ".join(cmd), flush=True)
        res = subprocess.run(cmd, capture_output=True, text=True)
        out = "\n".join(l for l in (res.stdout + res.stderr).splitlines()
                        if "packed-fp32-ops" not in l)
        if res.returncode != 0:
            raise RuntimeError("hipcc failed:\n" + out)
        if verbose and out.strip():
            print(out)

    tmp = LIB + ".tmp"
    with tempfile.TemporaryDirectory() as objs, concurrent.futures.ThreadPoolExecutor(8) as pool:
        out = [os.path.join(objs, os.path.basename(f) + ".o") for f in sources]
        list(pool.map(run, [flags + ["-c", f, "-o", o] for f, o in zip(sources, out)]))
        run([hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC"] + out + ["-o", tmp])
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
