"""Build libzero.so (the C-ABI library) for gfx950 with hipcc, in-tree."""
import os
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libzero.so")
SOURCES = [os.path.join(CSRC, f) for f in ("zero_kernels.hip", "zero_api.cpp", "zero_ops.hip", "zero_ops_api.cpp",
                                              "zero_linear.hip", "zero_muon.hip", "zero_hidden_api.cpp")]

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
# -ffp-contract=off: one rounding per fp32 operation (no fused multiply-add).
# -packed-fp32-ops off: no v_pk_* fp32 instructions are generated.
FLAGS = ["--offload-arch=gfx950", "-O3", "-std=c++17", "-ffp-contract=off", "-fno-fast-math",
         "-fPIC", "-fvisibility=hidden", "-Wall",
         "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
         "-I" + INCLUDE, "-I" + CSRC]


def build(force=True):
    if not force and os.path.exists(LIB):
        return LIB
    tmp = LIB + ".tmp"
    with tempfile.TemporaryDirectory() as objects:
        def run(cmd):
            return subprocess.run([HIPCC, *FLAGS, *cmd], capture_output=True, text=True)

        objs = [os.path.join(objects, os.path.basename(s) + ".o") for s in SOURCES]
        with ThreadPoolExecutor(min(len(SOURCES), os.cpu_count() or 1)) as pool:
            done = list(pool.map(lambda so: run(["-c", so[0], "-o", so[1]]), zip(SOURCES, objs)))
        done.append(run(["-shared", *objs, "-o", tmp]) if not any(r.returncode for r in done) else done[0])
        for r in done:
            if r.returncode != 0:
                sys.stderr.write(r.stdout + r.stderr)
                raise RuntimeError("hipcc failed building libzero.so")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build())
