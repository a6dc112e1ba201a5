"""Positions of tokens as the kernels compute them, compiled for the host and run against 64-bit arithmetic (no GPU)."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_positions(tmp_path):
    if subprocess.run(["which", "hipcc"], capture_output=True).returncode != 0:
        pytest.skip("hipcc is not installed")
    exe = str(tmp_path / "attn_places")
    r = subprocess.run(["hipcc", "-O2", "-std=c++17", "--offload-arch=gfx950", "-Xclang", "-target-feature", "-Xclang",
                        "-packed-fp32-ops", "-Xarch_host", "-fsanitize=undefined", "-Xarch_host",
                        "-fno-sanitize-recover=undefined", os.path.join(ROOT, "tests", "csrc", "attn_places.hip"), "-o", exe],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "ok" in r.stdout, r.stdout + r.stderr
