"""What a paged attention CTA does after a wait ran out: every request whose rows are then not written is flagged.
No wait is made to run out on a GPU; the walk over the tiles is host code too, and is run here."""
import os
import re
import subprocess

import pytest

from draft_tree_build_gb300 import _build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_a_cta_that_gives_up_reports_every_unit_it_leaves(tmp_path):
    exe = str(tmp_path / "paged_walk")
    r = subprocess.run([_build.nvcc(), "-O2", "-std=c++17", "-I", _build.CSRC, "-I", _build.INCLUDE,
                        os.path.join(ROOT, "tests", "host", "paged_walk.cu"), "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout


@pytest.mark.parametrize("text", [
    # the softmax warps, which write a unit's outputs, report what they leave unwritten ...
    r"if \(w\.left > 0\) leave\(w, c\.Hkv, a\.status, a\.acc \? a\.lse2 : nullptr, a\.G, kt\);",
    r"give_up\(w, heads, \[&\]\(int r, int g\) \{\s*if \(kt == 0\) atomicOr\(&status\[r\], BASTION_STATUS_TIMEOUT\);"
    r"\s*if \(lse2 && kt < G\) lse2\[[^;]*\] = INFINITY;",
    # ... and the weights of such a row are left as they were
    r"if \(isinf\(y\[h\]\)\) continue;",
])
def test_the_kernels_use_it(text):
    src = open(os.path.join(_build.CSRC, "paged_attention.cu")).read()
    assert len(re.findall(text, src)) == 1
