"""What no kernel source may hold."""
import glob
import os

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_no_multicast_into_clusters():
    """The benchmark runs this library on several GPUs at once: no copy or commit multicasts into a cluster, not even
    as an option."""
    files = [f for ext in ("cu", "cuh", "h", "c") for f in glob.glob(os.path.join(ROOT, "draft_tree_build_gb300", "csrc", "*." + ext))]
    assert len(files) > 15
    for f in files:
        text = open(f).read()
        assert "multicast::cluster" not in text, f
        assert "BASTION_LMHEAD_CLUSTER" not in text, f
