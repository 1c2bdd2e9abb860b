"""The operators on the hidden matrices at the ends of what the header allows,
without a GPU."""
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
def test_limits(tmp_path):
    """Calls of the largest sizes with stand-ins for the launchers: none within the
    header's limits is refused, and every launch has work and fits a grid
    (tests/native/hidden_limits.cpp)."""
    exe = tmp_path / "hidden_limits"
    csrc = os.path.join(ROOT, "zero_sharded_mixed_02_amd", "csrc")
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=undefined", "-Wall",
           "-Werror", "-I", os.path.join(ROOT, "include"), "-I", csrc, os.path.join(ROOT, "tests", "native", "hidden_limits.cpp"),
           os.path.join(csrc, "zero_api.cpp"), os.path.join(csrc, "zero_hidden_api.cpp"), "-o", str(exe)]
    subprocess.run(cmd, check=True, capture_output=True, text=True)
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:verify_asan_link_order=0")
    r = subprocess.run([str(exe)], capture_output=True, text=True, env=env, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    assert " 0 failures" in r.stdout


@pytest.mark.skipif(not os.path.exists("/opt/rocm/bin/hipcc"), reason="hipcc not available")
def test_small_matrices_registers():
    """The kernels of an orthogonalisation keep their values in registers: what the
    compiler reports of scratch stays below 64 bytes a lane (704 once made 128
    matrices of 128 x 128 take 100 us in place of 61)."""
    from zero_sharded_mixed_02_amd import _build
    cmd = [_build.HIPCC, *_build.FLAGS, "--cuda-device-only", "-c", os.path.join(_build.CSRC, "zero_muon.hip"), "-o", os.devnull,
           "-Rpass-analysis=kernel-resource-usage"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    sizes = [int(x) for x in re.findall(r"ScratchSize \[bytes/lane\]: (\d+)", r.stderr)]
    assert len(sizes) > 30 and max(sizes) < 64, sizes
