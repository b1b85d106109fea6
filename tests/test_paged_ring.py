"""What the warps that fill a shared-prefix attention CTA's ring wait for: host code too, and run here with each warp in turn
held up.  Nothing is made to wait on a GPU."""
import os
import subprocess

import pytest

from draft_tree_build_gb300 import _build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def model(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("ring") / "paged_ring")
    r = subprocess.run([_build.nvcc(), "-O2", "-std=c++17", "-Xcompiler", "-pthread", "-I", _build.CSRC,
                        os.path.join(ROOT, "tests", "host", "paged_ring.cu"), "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    return exe


def test_every_share_comes_to_its_end(model):
    """However late a warp begins: no phase passes that a warp has yet to look for."""
    r = subprocess.run([model], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout


def test_the_model_finds_a_phase_that_is_missed(model):
    """The values waiting for the first phase of the keys' own barrier, late: it has gone two phases on."""
    r = subprocess.run([model, "shared"], capture_output=True, text=True, timeout=300)
    assert r.returncode == 1 and "4 stages, 3 tiles, thread 1 late: stuck" in r.stdout, r.stdout
    assert "8 stages, 5 tiles, thread 1 late: stuck" in r.stdout, r.stdout
