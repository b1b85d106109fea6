"""The prefix launch of shared-prefix attention begins while the launch before it runs, and waits for it only at its end."""
import os
import re

from draft_tree_build_gb300 import _build


def _text(name):
    return re.sub(r"//[^\n]*", "", open(os.path.join(_build.CSRC, name)).read())


def test_the_groups_are_read_past_l1():
    """What other launches may have written just before: in L2 for certain, in this SM's L1 perhaps as it was."""
    body = _text("paged_prefix.cu")
    body = body[body.index("griddep_launch_dependents();"):body.index("griddep_wait();")]
    for name in ("start", "len", "table"):
        reads = re.findall(r"\ba\.%s\b" % name, body)
        assert reads and len(reads) == len(re.findall(r"__ldcg\(a\.%s\b" % name, body)), name
    for name in ("q", "seq_len", "own", "own_lse"):  # the own slots' launch has those
        assert not re.search(r"\ba\.%s\b" % name, body), name
    assert "c.table" not in body


def test_the_launch_before_it_waits_first():
    """It lets the prefix launch begin, which counts on everything before it being complete."""
    for name in ("paged_attention.cu", "paged_prefix_own.cu"):
        body = _text(name)
        first = body.index("griddep_launch_dependents();")
        assert body.rfind("griddep_wait();", 0, first) >= 0
        assert not body[body.rfind("griddep_wait();", 0, first) + len("griddep_wait();"):first].strip()
