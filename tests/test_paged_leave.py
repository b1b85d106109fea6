"""What shared-prefix attention's softmax warps report after a wait ran out, whichever of them stop, and where: a model on the
host, over the walk that the kernel has.  No wait is made to run out on a GPU."""
import os
import re
import subprocess

import pytest

from draft_tree_build_gb300 import _build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def model(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("leave") / "paged_leave")
    r = subprocess.run([_build.nvcc(), "-O2", "-std=c++17", "-I", _build.CSRC, "-I", _build.INCLUDE,
                        os.path.join(ROOT, "tests", "host", "paged_leave.cu"), "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    return exe


def test_every_request_that_is_left_is_told(model):
    r = subprocess.run([model], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout


def test_the_model_finds_a_request_that_is_not(model):
    """A warp that gives up alone and flags its own rows' share of the requests."""
    r = subprocess.run([model, "share"], capture_output=True, text=True, timeout=300)
    assert r.returncode == 1 and "nobody is told" in r.stdout


def test_the_kernel_does_as_the_model():
    """All four quarters of the requests, from where the warp stopped."""
    src = open(os.path.join(_build.CSRC, "paged_prefix.cu")).read()
    assert re.search(r"const Units<true> stop = w;\s*#pragma unroll 1\s*for \(int k = 0; k < 4; \+\+k\) \{\s*"
                     r"const int row = 32 \* k \+ lane;\s*Units<true> w = stop;\s*if \(!ok\)", src)
