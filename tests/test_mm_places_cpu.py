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


def plans(tmp_path, calls):
    """(kernel, shares of k) that the library chooses for each call (T, N, K, results)."""
    exe = host_program(tmp_path, "mm_plan")
    args = [str(int(v)) for T, N, K, ot in calls for v in (T, N, K, ot == "f32")]
    r = subprocess.run([exe, *args], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stderr
    return [(p.split()[0], int(p.split()[1])) for p in r.stdout.splitlines()]


def test_every_kernel_is_tested(tmp_path):
    """The GPU tests' sizes reach every kernel: with one share and with several, with tiles that end early, for both kinds of results; and
    the 8-bit instruction's kernels with every code, NaN and infinite scales."""
    from test_mm_exact_gpu import EXACT, VALUES
    tiles = dict(few=(16, 16), some32=(64, 32), some64=(64, 64), some128=(64, 128), tile128=(128, 128), tile256=(256, 256))
    seen = {}
    for (T, N, K, ot), (how, ks) in zip(EXACT, plans(tmp_path, EXACT)):
        n, t = tiles[how]
        seen.setdefault((how, ot == "f32"), []).append((ks, N % n != 0, T % t != 0, K % 128 != 0))
    for how in tiles:
        for f32 in (False, True):
            if (how, f32) == ("tile256", True):
                continue                                       # (fp32 results take the smaller tile)
            got = seen[how, f32]
            assert f32 or (any(ks == 1 for ks, *_ in got) and (how == "few" or any(ks > 1 for ks, *_ in got))), (how, got)
            assert any(n and t and k for _, n, t, k in got), (how, f32, got)
    for how in ("some128", "tile128"):
        assert any(ks > 1 for ks, *_ in seen[how, True]), how
    assert {"few", "some32", "some64", "some128", "tile128", "tile256"} == {how for how, _ in plans(tmp_path, VALUES)}
