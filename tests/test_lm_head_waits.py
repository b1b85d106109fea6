"""What the LM-head kernel does after a wait ran out, read in its source: no wait is made to run out on a GPU."""
import os
import re

from draft_tree_build_gb300 import _build


def test_an_lm_head_tile_that_gives_up_flags_all_of_its_rows():
    """A tile's 128 rows belong to several requests: the epilogue, a thread a row, flags each one's."""
    src = open(os.path.join(_build.CSRC, "lm_head_topk.cu")).read()
    wait = r"if \(!__all_sync\(kFull, wait_bar\(&bs\.acc_full\[buf\][^{;]*\) \{\s*//[^\n]*\n"
    assert len(re.findall(wait + r"\s*if \(live\) atomicOr\(&a\.status\[row / a\.b\], BASTION_STATUS_TIMEOUT\);\s*break;", src)) == 1
