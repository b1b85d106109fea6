"""The page plan whose positions begin behind a prefix: the C ABI's host checks (fake pointers, never dereferenced) and the
binding's."""
import ctypes

import pytest
import torch

from test_layer_refusals import PLAN, _marshal_calls, _plan_args
from test_paged_refusals import NULL, SIZE, UNSUPPORTED, WORKSPACE, _Fake, b  # noqa: F401

vp = ctypes.c_void_p


def _plan(b, offset=vp(0x900000), **over):  # noqa: F811
    assert set(over) <= set(PLAN)
    args = list({**PLAN, **over}.values())
    return b.lib().bastion_paged_plan_offset(*args[:-4], offset, *args[-4:])


def test_the_offset_is_needed(b):  # noqa: F811
    assert _plan(b, None) == NULL
    assert _plan(b, B=0) == SIZE


@pytest.mark.parametrize("at", [0x100000, 0x100000 + 4 * 4 * 20 - 4, 0x200000, 0x220008, 0x230000 - 12, 0x300000, 0x400000 + 252,
                                0x500000, 0x700000, 0x900000])
def test_no_output_lies_over_it(b, at):  # noqa: F811
    """Table, lengths, pages held, free list and its count, slots, positions, status, row starts."""
    packed = dict(start=vp(0x900000)) if at == 0x900000 else {}
    assert _plan(b, vp(at), ws_bytes=0, **packed) == UNSUPPORTED


@pytest.mark.parametrize("at", [0x210000, 0x100000 + 4 * 4 * 20, 0x200010, 0x900000])
def test_apart(b, at):  # noqa: F811
    """The counts of new tokens are an input, too."""
    assert _plan(b, vp(at), ws_bytes=0) == WORKSPACE


@pytest.mark.parametrize("bad", [torch.zeros(3, dtype=torch.int32), torch.zeros(4), torch.zeros(4, 1, dtype=torch.int32)])
def test_binding(b, bad):  # noqa: F811
    with pytest.raises(b.BastionError, match="pos_offset"):
        b.bastion_paged_plan(**_plan_args(), pos_offset=bad)
    with pytest.raises(b.BastionError, match="CUDA device"):
        b.bastion_paged_plan(**_plan_args(), pos_offset=torch.zeros(4, dtype=torch.int32))


def test_short_way(b):  # noqa: F811
    """Eighteen arguments go to the one entry point, nineteen with a tensor to the other; what is no offset is declined."""
    m = b._marshal
    zero = ctypes.cast(ctypes.pythonapi.PyGILState_Check, vp).value  # 0: the interpreter's lock is not held
    one = ctypes.CFUNCTYPE(ctypes.c_int)(lambda: 1)
    try:
        m.init(torch.bfloat16, torch.float16, torch.float32, torch.int32, torch.uint8, lambda: 0, lambda dev: 0, zero, zero, zero)
        m.init_layer(torch.int64, torch.float64, zero, zero, zero)
        m.init_offset(ctypes.cast(one, vp).value)
        (f, args), _, _ = _marshal_calls(b, _Fake)
        four = _Fake(torch.zeros(4, dtype=torch.int32))
        assert f(*args) == 0 and f(*args, None) == 0 and f(*args, four) == 1
        for bad in (3, "x", args[0], _Fake(torch.zeros(4)), _Fake(torch.zeros(5, dtype=torch.int32))):
            assert f(*args, bad) is None
        assert f(*args, None, None) is None
    finally:
        b._marshal = b._load_marshal(b.lib())


def test_the_cache_passes_it_on(b, monkeypatch):  # noqa: F811
    seen = []
    monkeypatch.setattr(b, "bastion_paged_plan", lambda *a: seen.append(a))
    c, offset = b.PagedCache(2, 4, 2, 64, 8, 4, "cpu", new_tokens=3), torch.zeros(2, dtype=torch.int32)
    c.reserve(3, pos_offset=offset)
    c.reserve(3)
    assert seen[0][-1] is offset and seen[1][-1] is None
