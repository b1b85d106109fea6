"""Refusals of the page plan, the norm and rotation and the shared-prefix attention: the C ABI's host checks (fake
pointers, never dereferenced: every call fails before a launch) and the binding's."""
import ctypes

import pytest
import torch

from test_paged_refusals import ALIGN, CACHE_REFUSALS, DTYPE, NULL, SIZE, UNSUPPORTED, WORKSPACE, _struct, b, vp  # noqa: F401

cf = ctypes.c_float
PLAN = dict(table=vp(0x100000), B=4, max_pages=20, page=16, n_pages=100, seq_len=vp(0x200000), n_new=vp(0x210000), m=8,
            seq_len_out=vp(0x200000), held=vp(0x220000), held_out=vp(0x220000), stack=vp(0x300000), n_free=vp(0x230000),
            n_free_out=vp(0x230000), trim=0, slots=vp(0x400000), pos=vp(0x500000), n_rows=32, start=None, ws=vp(0x600000),
            ws_bytes=1 << 20, status=vp(0x700000), stream=None)
ROPE = dict(dtype=1, T=10, Hq=8, Hkv=2, D=128, q=vp(0x100000), qt=12 * 128, qh=128, k=vp(0x100000 + 8 * 256), kt=12 * 128,
            kh=128, v=None, vt=0, vh=0, qw=vp(0x200000), kw=vp(0x210000), eps=cf(1e-6), pos=vp(0x220000),
            freq=vp(0x230000), rot=128, inter=0, factor=cf(1.0), qo=vp(0x300000), qot=1024, qoh=128, ko=vp(0x400000),
            kot=256, koh=128, cache=None, slots=None, status=vp(0x500000), stream=None)
ATTEND = dict(pt=vp(0x800000), pages=100, plen=vp(0x810000), start=vp(0x820000), groups=3, q=vp(0x400000), Hq=32,
              q_stride=32 * 128, seq_len=vp(0x500000), scale=cf(0.1), out=vp(0x600000), lse=vp(0x700000),
              ws=vp(0xa00000), ws_bytes=1 << 30, status=vp(0xb00000), stream=None)


def _plan(b, **over):  # noqa: F811
    assert set(over) <= set(PLAN)
    return b.lib().bastion_paged_plan(*{**PLAN, **over}.values())


@pytest.mark.parametrize("over,code", [
    *[({n: None}, NULL) for n in ("table", "seq_len", "held", "held_out", "stack", "n_free", "n_free_out", "slots", "pos",
                                  "ws", "status")],
    (dict(B=0), SIZE), (dict(B=1025), SIZE), (dict(max_pages=0), SIZE), (dict(max_pages=(1 << 24) + 1), SIZE),
    (dict(n_pages=0), SIZE), (dict(n_pages=1 << 31), SIZE), (dict(m=0), SIZE), (dict(m=321), SIZE), (dict(n_rows=31), SIZE),
    (dict(n_rows=33), SIZE), (dict(n_rows=0, start=vp(0x800000)), SIZE), (dict(n_rows=1 << 31, start=vp(0x800000)), SIZE),
    (dict(page=0), SIZE), (dict(page=-16), SIZE), (dict(page=4), UNSUPPORTED), (dict(page=24), UNSUPPORTED),
    (dict(page=256, max_pages=4), UNSUPPORTED), (dict(ws=vp(0x600010)), ALIGN), (dict(slots=vp(0x400004)), ALIGN),
    (dict(pos=vp(0x500002)), ALIGN), (dict(ws_bytes=64), WORKSPACE), (dict(seq_len_out=vp(0x200004)), UNSUPPORTED),
    (dict(held_out=vp(0x21fffc)), UNSUPPORTED), (dict(n_free_out=vp(0x220000)), UNSUPPORTED),
    (dict(held_out=vp(0x200000)), UNSUPPORTED), (dict(seq_len_out=vp(0x220000)), UNSUPPORTED),
    (dict(seq_len_out=vp(0x210000)), UNSUPPORTED), (dict(held_out=vp(0x210008)), UNSUPPORTED),
    (dict(slots=vp(0x300000)), UNSUPPORTED), (dict(pos=vp(0x400000)), UNSUPPORTED), (dict(pos=vp(0x100000)), UNSUPPORTED),
    (dict(stack=vp(0x100010)), UNSUPPORTED), (dict(status=vp(0x20000c)), UNSUPPORTED),
    (dict(start=vp(0x230000)), UNSUPPORTED), (dict(start=vp(0x500000)), UNSUPPORTED),
    (dict(n_free=vp(0x300000)), UNSUPPORTED), (dict(status=vp(0x300000)), UNSUPPORTED),
])
def test_plan_refusals(b, over, code):  # noqa: F811
    assert _plan(b, **over) == code


def _rope(b, **over):  # noqa: F811
    assert set(over) <= set(ROPE)
    return b.lib().bastion_qk_norm_rope(*{**ROPE, **over}.values())


STORE = dict(v=vp(0x100000 + 10 * 256), vt=12 * 128, vh=128, slots=vp(0x240000))


@pytest.mark.parametrize("over,code", [
    *[({n: None}, NULL) for n in ("q", "k", "pos", "freq", "status", "qw", "kw")],
    (dict(qo=None, ko=None), NULL), (STORE, NULL), (dict(slots=vp(0x240000)), NULL), (dict(v=vp(0x800000)), NULL),
    (dict(dtype=0), DTYPE), (dict(dtype=3), DTYPE), (dict(T=0), SIZE), (dict(Hq=0), SIZE), (dict(Hkv=0), SIZE),
    (dict(D=0), SIZE), (dict(T=1 << 28), SIZE), (dict(Hq=65535), SIZE), (dict(D=256), UNSUPPORTED), (dict(D=96), UNSUPPORTED),
    (dict(rot=-16), SIZE), (dict(rot=144), SIZE), (dict(rot=8), SIZE), (dict(eps=cf(-1e-6)), SIZE),
    (dict(eps=cf(float("nan"))), SIZE), (dict(eps=cf(float("inf"))), SIZE), (dict(factor=cf(float("inf"))), SIZE),
    (dict(factor=cf(float("nan"))), SIZE), (dict(qt=1540), SIZE), (dict(qh=64), SIZE), (dict(kt=-256), SIZE),
    (dict(qot=1016), SIZE), (dict(kot=0), SIZE), (dict(koh=132), SIZE), (dict(q=vp(0x100008)), ALIGN),
    (dict(ko=vp(0x400002)), ALIGN), (dict(qw=vp(0x200008)), ALIGN), (dict(freq=vp(0x230004)), ALIGN),
    (dict(qo=vp(0x100000)), UNSUPPORTED),  # q's place with other strides
    (dict(qo=vp(0x100000 + 8 * 256), qot=12 * 128), UNSUPPORTED),  # k's rows
    (dict(qo=vp(0x100000 - 256), qot=12 * 128), UNSUPPORTED),  # a head further
    (dict(ko=vp(0x100000 + 9 * 256), kot=12 * 128), UNSUPPORTED), (dict(ko=vp(0x300000 + 512)), UNSUPPORTED),
    (dict(ko=vp(0x300000 + 2048), kot=1024), UNSUPPORTED), (dict(qo=vp(0x200000 - 128)), UNSUPPORTED),
    (dict(status=vp(0x300010)), UNSUPPORTED), (dict(status=vp(0x220000)), UNSUPPORTED), (dict(pos=vp(0x400000)), UNSUPPORTED),
])
def test_rope_refusals(b, over, code):  # noqa: F811
    assert _rope(b, **over) == code


@pytest.mark.parametrize("over,code", CACHE_REFUSALS)
def test_rope_cache_refusals(b, over, code):  # noqa: F811
    cache = dict(k_pool=0x10000000, v_pool=0x20000000, Hkv=2, stride_page=16 * 256, stride_slot=256) | over
    assert _rope(b, **STORE, cache=_struct(b, **cache)) == code


def test_rope_cache_of_another_shape(b):  # noqa: F811
    for over, code in ((dict(Hkv=4), SIZE), (dict(D=64), SIZE), (dict(dtype=2), DTYPE)):
        cache = dict(k_pool=0x10000000, v_pool=0x20000000, Hkv=2) | over
        assert _rope(b, **STORE, cache=_struct(b, **cache)) == code
    ok = dict(k_pool=0x10000000, v_pool=0x20000000, Hkv=2)
    for over, code in ((dict(v=vp(0x100008)), ALIGN), (dict(slots=vp(0x240004)), ALIGN), (dict(vt=4), SIZE),
                       (dict(qo=vp(0x100000 + 4 * 256), qot=12 * 128), UNSUPPORTED),
                       (dict(ko=vp(0x100000 + 10 * 256), kot=12 * 128), UNSUPPORTED), (dict(slots=vp(0x300000)), UNSUPPORTED)):
        assert _rope(b, **{**STORE, **over}, cache=_struct(b, **ok)) == code


def _attend(b, cache=None, **over):  # noqa: F811
    assert set(over) <= set(ATTEND)
    return b.lib().bastion_paged_prefix_attention(_struct(b, **(cache or {})), *{**ATTEND, **over}.values())


@pytest.mark.parametrize("over,code", CACHE_REFUSALS)
def test_prefix_cache_refusals(b, over, code):  # noqa: F811
    assert _attend(b, over) == code


@pytest.mark.parametrize("over,code", [
    *[({n: None}, NULL) for n in ("pt", "plen", "start", "q", "seq_len", "out", "ws", "status")],
    (dict(pages=0), SIZE), (dict(pages=(1 << 24) + 1), SIZE), (dict(groups=0), SIZE), (dict(groups=1025), SIZE),
    (dict(groups=1000, pages=1 << 22), SIZE), (dict(Hq=0), SIZE), (dict(Hq=33), SIZE), (dict(Hq=136), UNSUPPORTED),
    (dict(scale=cf(0.0)), SIZE), (dict(scale=cf(float("nan"))), SIZE), (dict(scale=cf(float("inf"))), SIZE),
    (dict(q_stride=4100), SIZE), (dict(q_stride=-4096), SIZE), (dict(q_stride=0), SIZE), (dict(q_stride=4088), SIZE), (dict(q=vp(0x400008)), ALIGN), (dict(out=vp(0x600002)), ALIGN),
    (dict(ws=vp(0xa00010)), ALIGN), (dict(pt=vp(0x800002)), ALIGN), (dict(ws_bytes=1000), WORKSPACE),
    (dict(out=vp(0x400000), q_stride=8192), UNSUPPORTED), (dict(out=vp(0x400010)), UNSUPPORTED),
    (dict(lse=vp(0x600000)), UNSUPPORTED), (dict(lse=vp(0x400100)), UNSUPPORTED), (dict(lse=vp(0x81fffc)), UNSUPPORTED),
    (dict(status=vp(0x800010)), UNSUPPORTED), (dict(status=vp(0x500000)), UNSUPPORTED), (dict(status=vp(0x700004)), UNSUPPORTED),
    (dict(plen=vp(0x600100)), UNSUPPORTED), (dict(start=vp(0x700010)), UNSUPPORTED),
])
def test_prefix_refusals(b, over, code):  # noqa: F811
    assert _attend(b, **over) == code


def test_workspace_queries(b):  # noqa: F811
    L = b.lib()
    assert L.bastion_paged_plan_workspace_bytes(0) == 0 == L.bastion_paged_plan_workspace_bytes(1025)
    assert L.bastion_paged_plan_workspace_bytes(1024) > 0
    size = L.bastion_paged_prefix_attention_workspace_bytes
    assert size(64, 32, 8, 128, 1) > 0
    for bad in ((0, 32, 8, 128, 1), (1025, 32, 8, 128, 1), (4, 33, 8, 128, 1), (4, 136, 8, 128, 1), (4, 32, 8, 96, 1),
                (4, 32, 8, 128, 0), (4, 32, 8, 128, 1025)):
        assert size(*bad) == 0
    for code in (b.STATUS_NO_PAGE, b.STATUS_BAD_GROUP):
        assert b.bastion_status_string(code) != "unknown code"


# --------------------------------------------------------------------------- the binding's checks, on CPU tensors

i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731


def _plan_args():
    return dict(page_table=i32(4, 20), page_size=16, seq_len=i32(4), m=8, held=i32(4), held_out=i32(4),
                free_pages=i32(100), n_free=i32(1), n_free_out=i32(1), slots=torch.zeros(32, dtype=torch.int64), pos=i32(32),
                workspace=torch.zeros(4096, dtype=torch.uint8), status=i32(4))


@pytest.mark.parametrize("over,match", [
    (dict(page_table=i32(80)), "page_table"), (dict(page_table=i32(4, 20).long()), "page_table"),
    (dict(page_table=i32(20, 4).T), "page_table"), (dict(seq_len=i32(5)), "seq_len"), (dict(held=i32(4).long()), "held"),
    (dict(held_out=i32(3)), "held_out"), (dict(n_new=i32(3)), "n_new"), (dict(n_free=i32(2)), "n_free"),
    (dict(n_free_out=torch.zeros(1)), "n_free_out"), (dict(free_pages=i32(10, 10)), "free_pages"), (dict(slots=i32(32)), "slots"),
    (dict(pos=i32(31)), "pos"), (dict(row_start=i32(4)), "row_start"), (dict(status=i32(4, 1)), "status"),
    (dict(m=1 << 32), "32 bits"), (dict(page_size=1 << 40), "32 bits"), (dict(workspace=i32(1024)), "workspace"), ({}, "CUDA device"),
])
def test_plan_binding(b, over, match):  # noqa: F811
    with pytest.raises(b.BastionError, match=match):
        b.bastion_paged_plan(**{**_plan_args(), **over})


def _rope_args():
    return dict(q=bf(10, 8, 128), k=bf(10, 2, 128), pos=i32(10), inv_freq=torch.ones(64, dtype=torch.float64),
                q_out=bf(10, 8, 128), status=i32(1), k_out=bf(10, 2, 128), q_weight=bf(128), k_weight=bf(128))


POOLS = dict(v=bf(10, 2, 128), k_pool=bf(5, 16, 2, 128), v_pool=bf(5, 16, 2, 128), slots=torch.zeros(10, dtype=torch.int64))


@pytest.mark.parametrize("over,match", [
    (dict(q=bf(10, 1024)), "must be"), (dict(q=torch.zeros(10, 8, 128)), "bfloat16 or float16"), (dict(k=bf(9, 2, 128)), "k must"),
    (dict(k=bf(10, 2, 64)), "k must"), (dict(k=bf(10, 128, 2).transpose(1, 2)), "k must"), (dict(q_out=bf(10, 8, 64)), "q_out"),
    (dict(k_out=bf(10, 2, 128).half()), "k_out"), (dict(pos=i32(11)), "pos"), (dict(pos=i32(10).long()), "pos"),
    (dict(inv_freq=torch.ones(64)), "inv_freq"), (dict(inv_freq=torch.ones(8, 8, dtype=torch.float64)), "inv_freq"),
    (dict(q_weight=bf(64)), "q_weight"), (dict(k_weight=torch.ones(128)), "k_weight"), (dict(status=i32(10)), "status"),
    ({**POOLS, "slots": i32(10)}, "slots"), ({**POOLS, "v_pool": None}, "together"), ({**POOLS, "v": bf(10, 3, 128)}, "v must"),
    ({**POOLS, "k_pool": bf(5, 16, 2, 128).half()}, "pools"), ({**POOLS, "k_pool": bf(5, 2, 16, 128).transpose(1, 2)}, "pools"),
    ({}, "CUDA device"), (POOLS, "CUDA device"),
])
def test_rope_binding(b, over, match):  # noqa: F811
    with pytest.raises(b.BastionError, match=match):
        b.bastion_qk_norm_rope(**{**_rope_args(), **over})


def _prefix_args():
    return dict(q=bf(4, 8, 128), k_pool=bf(9, 16, 2, 128), v_pool=bf(9, 16, 2, 128), page_table=i32(4, 3), seq_len=i32(4),
                prefix_table=i32(2, 5), prefix_len=i32(2), group_start=i32(3), scale=0.1, out=bf(4, 8, 128),
                workspace=torch.zeros(4096, dtype=torch.uint8), status=i32(4), lse=torch.zeros(4, 8))


@pytest.mark.parametrize("over,match", [
    (dict(q=bf(4, 8, 64)), "q must"), (dict(q=bf(3, 8, 128)), "q must"), (dict(q=bf(4, 8, 128).half()), "q must"),
    (dict(q=bf(4, 128, 8).transpose(1, 2)), "heads of q"), (dict(out=bf(4, 8, 64)), "out"), (dict(lse=torch.zeros(8, 4)), "lse"),
    (dict(prefix_table=i32(10)), "prefix_table"), (dict(prefix_table=i32(2, 5).long()), "prefix_table"),
    (dict(prefix_len=i32(3)), "prefix_len"), (dict(group_start=i32(2)), "group_start"), (dict(seq_len=i32(5)), "seq_len"),
    (dict(page_table=i32(4, 3).long()), "page_table"), (dict(workspace=i32(8)), "workspace"), ({}, "CUDA device"),
])
def test_prefix_binding(b, over, match):  # noqa: F811
    with pytest.raises(b.BastionError, match=match):
        b.bastion_paged_prefix_attention(**{**_prefix_args(), **over})


def test_rope_frequencies(b):  # noqa: F811
    f, size = b.rope_frequencies(128, 10000.0, "cpu")
    assert size == 1.0 and f.dtype == torch.float64 and f.shape == (64,) and float(f[0]) == 1.0
    assert float(f[32]) == pytest.approx(0.01)
    assert torch.allclose(b.rope_frequencies(128, 10000.0, "cpu", "linear", 4.0)[0], f / 4)
    g = b.rope_frequencies(128, 10000.0, "cpu", "base", 4.0)[0]
    assert float(g[0]) == 1.0 and float(g[-1]) == pytest.approx(float(f[-1]) / 4)
    g = b.rope_frequencies(128, 5e5, "cpu", "bands", 8.0)[0]
    f = b.rope_frequencies(128, 5e5, "cpu")[0]
    turns = 8192 * f / 6.283185307179586
    assert torch.equal(g[turns > 4], f[turns > 4]) and torch.allclose(g[turns < 1], f[turns < 1] / 8)
    mid = (turns > 1) & (turns < 4)
    assert bool(mid.any()) and bool(((g < f) & (g > f / 8))[mid].all())
    g, size = b.rope_frequencies(128, 5e5, "cpu", "yarn", 8.0, low=1.0, high=32.0)
    assert size == pytest.approx(0.1 * 2.0794415416798357 + 1) and float(g[0]) == 1.0
    assert float(g[-1]) == pytest.approx(float(f[-1]) / 8)
    with pytest.raises(b.BastionError, match="scaling"):
        b.rope_frequencies(128, scaling="other")


# --------------------------------------------------------------------------- the compiled short way

def _marshal_calls(b, wrap=lambda t: t):  # noqa: F811
    w = {n: wrap(x) if isinstance(x, torch.Tensor) else x for args in (_plan_args(), {}) for n, x in args.items()}
    plan = [w[n] for n in ("page_table", "page_size", "seq_len", "m", "held", "held_out", "free_pages", "n_free", "n_free_out",
                           "slots", "pos", "workspace", "status")] + [None, None, None, False, None]
    r = {n: wrap(x) for n, x in {**_rope_args(), **POOLS}.items()}
    rope = [r["q"], r["k"], r["pos"], r["inv_freq"], r["q_out"], r["status"], r["k_out"], r["q_weight"], r["k_weight"], 1e-6,
            False, 1.0, r["v"], r["k_pool"], r["v_pool"], r["slots"], None]
    p = {n: wrap(x) if isinstance(x, torch.Tensor) else x for n, x in _prefix_args().items()}
    prefix = [p[n] for n in ("q", "k_pool", "v_pool", "page_table", "seq_len", "prefix_table", "prefix_len", "group_start",
                             "scale", "out", "workspace", "status")] + [None, None]
    return (b._marshal.plan, plan), (b._marshal.rope, rope), (b._marshal.prefix, prefix)


def test_marshal_declines_what_the_binding_refuses(b):  # noqa: F811
    """CPU tensors, too few and too many arguments, and anything odd in any place: nothing is called."""
    assert b._marshal is not None
    for f, args in _marshal_calls(b):
        assert f(*args) is None
        assert f() is None and f(*args, None) is None
        for i in range(len(args)):
            for bad in (None, 3, "x", 1 << 70, torch.zeros(1, 1, 1, 1, 1), object()):
                assert f(*args[:i], bad, *args[i + 1:]) is None


class _Fake:
    """What the short way looks at of a tensor; on device 0."""

    def __init__(self, t):
        self.t, self.dtype, self.shape = t, t.dtype, tuple(t.shape)
        self.stride, self.is_contiguous, self.data_ptr = t.stride, t.is_contiguous, t.data_ptr

    def get_device(self):
        return 0


def test_marshal_calls_without_the_interpreters_lock(b):  # noqa: F811
    """A function that says whether its thread holds the lock, in place of the library's; and wrong arguments on a GPU's
    tensors are declined, too."""
    m = b._marshal
    held = ctypes.cast(ctypes.pythonapi.PyGILState_Check, vp).value
    try:
        m.init(torch.bfloat16, torch.float16, torch.float32, torch.int32, torch.uint8, lambda: 0, lambda dev: 0, held, held,
               held)
        m.init_layer(torch.int64, torch.float64, held, held, held)
        for f, args in _marshal_calls(b, _Fake):
            assert f(*args) == 0
            for i, x in enumerate(args):
                if isinstance(x, _Fake):
                    for bad in (_Fake(x.t.double() if x.dtype is not torch.float64 else x.t.float()), _Fake(x.t[..., None]),
                                _Fake(torch.cat([x.t, x.t], -1)), 3):
                        # one dimension of the free list, the table, the workspace, the rows or the frequencies is free
                        got = f(*args[:i], bad, *args[i + 1:])
                        assert got is None or not isinstance(bad, int) and bad.dtype is x.dtype and len(bad.shape) == len(x.shape)
        (f, plan), (g, rope), _ = _marshal_calls(b, _Fake)
        assert f(*plan[:1], 1 << 40, *plan[2:]) is None and f(*plan[:3], 8.0, *plan[4:]) is None
        assert g(*rope[:13], None, *rope[14:]) is None and g(*rope[:9], "eps", *rope[10:]) is None
        m.init(torch.bfloat16, torch.float16, torch.float32, torch.int32, torch.uint8, lambda: 1, lambda dev: 0, held, held,
               held)
        for f, args in _marshal_calls(b, _Fake):
            assert f(*args) is None  # another device is current
    finally:
        b._marshal = b._load_marshal(b.lib())
