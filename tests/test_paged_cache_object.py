"""PagedCache's own buffers, on the CPU."""
import pytest
import torch


@pytest.mark.parametrize("kw", [{}, dict(weights=True), dict(new_tokens=3), dict(prefixes=2), dict(new_tokens=3, prefixes=2)])
def test_all_workspaces_are_cleared(kw):
    """After a wait that ran out: whichever call it was, its workspace is among them."""
    from draft_tree_build_gb300 import bastion
    c = bastion.PagedCache(2, 4, 2, 64, 8, 4, "cpu", **kw)
    spaces = {n: x for n, x in vars(c).items() if isinstance(x, torch.Tensor) and x.dtype == torch.uint8}
    assert len(spaces) == 2 + sum(map(bool, (kw.get("weights"), kw.get("new_tokens"), kw.get("prefixes"))))
    before = {n: x.clone() for n, x in vars(c).items() if isinstance(x, torch.Tensor) and n not in spaces}
    for x in spaces.values():
        x.fill_(3)
    c.clear_workspaces()
    for n, x in spaces.items():
        assert not bool(x.any()), n
    for n, x in before.items():
        assert torch.equal(getattr(c, n), x), n
