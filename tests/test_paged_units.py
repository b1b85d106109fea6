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


def test_a_cta_that_gives_up_reports_what_it_leaves():
    """No wait is made to run out on a GPU: the softmax warps, which write the parts, flag every request of the tiles
    that are left, the current segment's among them."""
    import re
    src = open(os.path.join(_build.CSRC, "paged_prefix.cu")).read()
    assert len(re.findall(r"if \(!ok\) \{[^\n]*\n\s*for \(; w\.left > 0; w\.step\(c\.Hkv, a\.nb\)\)\s*"
                          r"for \(int b = w\.req \+ row; b < w\.req \+ w\.n; b \+= 128\) "
                          r"atomicOr\(&a\.status\[b\], BASTION_STATUS_TIMEOUT\);", src)) == 1
