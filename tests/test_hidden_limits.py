"""The operators on the hidden matrices at the ends of what the header allows,
without a GPU."""
import os
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
