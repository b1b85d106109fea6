"""Numbers that the paged cache's binding passes on: none is cut on its way."""
import pytest

from test_paged_refusals import _tensors, b  # noqa: F401


@pytest.mark.parametrize("kw", [dict(n_sink=-(1 << 32)), dict(n_recent=-(1 << 32) + 1), dict(budget=-(1 << 32) + 8),
                                dict(budget=-(1 << 31) - 1), dict(n_sink=1 << 32), dict(n_recent=1 << 31)])
def test_evict_counts_fit_32_bits(b, kw):  # noqa: F811
    t = _tensors()
    a = {**dict(budget=8, n_sink=0, n_recent=0), **kw}
    with pytest.raises(b.BastionError, match="32 bits"):
        b.bastion_paged_evict(t["k"], t["v"], t["table"], t["lens"], t["lens"].clone(), t["acc"], t["pos"], a["budget"],
                              a["n_sink"], a["n_recent"], t["lens"], t["acc"], t["pos"], t["ws"], t["st"])
