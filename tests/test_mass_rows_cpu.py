"""Which new tokens a tile of keys takes in the attention mass, compiled for the host and run against brute force (no GPU)."""
import subprocess

from test_mm_places_cpu import host_program


def test_rows(tmp_path):
    r = subprocess.run([host_program(tmp_path, "mass_rows")], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "ok" in r.stdout, r.stdout + r.stderr
