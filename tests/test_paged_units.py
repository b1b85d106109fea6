"""How shared-prefix attention deals its tiles to CTAs and finds a row's parts again: host code too, and run here."""
import os
import subprocess

from draft_tree_build_gb300 import _build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_every_tile_is_in_one_part_of_its_row(tmp_path):
    exe = str(tmp_path / "paged_units")
    r = subprocess.run([_build.nvcc(), "-O2", "-std=c++17", "-I", _build.CSRC, "-I", _build.INCLUDE,
                        os.path.join(ROOT, "tests", "host", "paged_units.cu"), "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout
