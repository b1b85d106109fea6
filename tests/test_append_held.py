"""Appending into the pages that requests hold: the C ABI's host checks (fake pointers, never dereferenced) and the binding's."""
import ctypes

import pytest
import torch

from test_paged_refusals import APPEND, CACHE_REFUSALS, NULL, UNSUPPORTED, WORKSPACE, _Fake, _struct, _tensors, b  # noqa: F401

vp = ctypes.c_void_p


def _call(b, held=vp(0xe00000), cache=None, **over):  # noqa: F811
    assert set(over) <= set(APPEND)
    return b.lib().bastion_paged_append_held(_struct(b, **(cache or {})), held, *{**APPEND, **over}.values())


@pytest.mark.parametrize("over,code", CACHE_REFUSALS)
def test_cache_refusals(b, over, code):  # noqa: F811
    assert _call(b, cache=over) == code


def test_held_is_needed(b):  # noqa: F811
    assert _call(b, held=None) == NULL


@pytest.mark.parametrize("held", [0x600000, 0x600000 - 12, 0x700004, 0x800000, 0x900010, 0xb00000, 0xb0000c])
def test_no_output_lies_over_it(b, held):  # noqa: F811
    """Lengths, counts, weights, positions, status."""
    assert _call(b, vp(held), ws_bytes=0) == UNSUPPORTED


@pytest.mark.parametrize("held", [0x600000 - 16, 0x600010, 0xb00010, 0xd00000])
def test_apart(b, held):  # noqa: F811
    assert _call(b, vp(held), ws_bytes=0) == WORKSPACE


@pytest.mark.parametrize("bad", [torch.zeros(3, dtype=torch.int32), torch.zeros(2), torch.zeros(2, 1, dtype=torch.int32)])
def test_binding(b, bad):  # noqa: F811
    t = _tensors()
    args = (t["new"], t["new"], t["k"], t["v"], t["table"], t["lens"], t["lens"], t["ws"], t["st"])
    with pytest.raises(b.BastionError, match="held"):
        b.bastion_paged_append(*args, held=bad)
    with pytest.raises(b.BastionError, match="CUDA device"):
        b.bastion_paged_append(*args, held=t["lens"].clone())


def test_short_way(b):  # noqa: F811
    """Sixteen arguments go to the one entry point, seventeen with a tensor to the other; what is not held's is declined."""
    m, t = b._marshal, {n: _Fake(x) for n, x in _tensors().items()}
    zero = ctypes.cast(ctypes.pythonapi.PyGILState_Check, vp).value  # 0: the interpreter's lock is not held
    one = ctypes.CFUNCTYPE(ctypes.c_int)(lambda: 1)
    args = [t["new"], t["new"], t["k"], t["v"], t["table"], t["lens"], t["lens"], t["ws"], t["st"], *[None] * 7]
    try:
        m.init(torch.bfloat16, torch.float16, torch.float32, torch.int32, torch.uint8, lambda: 0, lambda dev: 0, zero, zero, zero)
        m.init_held(ctypes.cast(one, vp).value)
        assert m.append(*args) == 0 and m.append(*args, None) == 0 and m.append(*args, t["lens"]) == 1
        for bad in (3, "x", t["table"], _Fake(torch.zeros(2)), _Fake(torch.zeros(3, dtype=torch.int32))):
            assert m.append(*args, bad) is None
        assert m.append(*args, None, None) is None
    finally:
        b._marshal = b._load_marshal(b.lib())


def test_the_cache_passes_what_its_requests_hold(b, monkeypatch):  # noqa: F811
    """PagedCache.append tells the pages held where the cache gives them out, and reserve(advance=False) no new lengths."""
    seen = []
    monkeypatch.setattr(b, "bastion_paged_append", lambda *a: seen.append(a))
    monkeypatch.setattr(b, "bastion_paged_plan", lambda *a: seen.append(a))
    own, plain = b.PagedCache(2, 4, 2, 64, 8, 4, "cpu", new_tokens=3), b.PagedCache(2, 4, 2, 64, 8, 4, "cpu")
    own.append(1, 2)
    plain.append(1, 2)
    assert seen[0][-1] is own.held and seen[1][-1] is None
    own.reserve(3, advance=False)
    own.reserve(3)
    lens = [[x is own.seq_len for x in a] for a in seen[2:]]
    assert [sum(x) for x in lens] == [1, 2]
