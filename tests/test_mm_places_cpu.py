"""Where the block-scaled product's kernels read, compiled for the host and run against brute force (no GPU)."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def host_program(tmp_path, name):
    """tests/csrc/<name>.hip as a host program under the undefined-behaviour sanitizer."""
    if subprocess.run(["which", "hipcc"], capture_output=True).returncode != 0:
        pytest.skip("hipcc is not installed")
    exe = str(tmp_path / name)
    r = subprocess.run(["hipcc", "-O2", "-std=c++17", "--offload-arch=gfx950", "-Xclang", "-target-feature", "-Xclang",
                        "-packed-fp32-ops", "-Xarch_host", "-fsanitize=undefined", "-Xarch_host",
                        "-fno-sanitize-recover=undefined", os.path.join(ROOT, "tests", "csrc", name + ".hip"), "-o", exe],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    return exe


def test_places(tmp_path):
    r = subprocess.run([host_program(tmp_path, "mm_places")], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "ok" in r.stdout, r.stdout + r.stderr
