"""Refusals of the paged cache's calls: the C ABI's host checks (fake pointers,
never dereferenced: every call fails before a launch) and the binding's."""
import ctypes
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NULL, SIZE, DTYPE, ALIGN, WORKSPACE, UNSUPPORTED = -1, -2, -3, -4, -5, -6
vp = ctypes.c_void_p


@pytest.fixture(scope="module")
def b():
    from draft_tree_build_gb300 import bastion
    bastion.lib()
    return bastion


def _declared():
    src = open(os.path.join(ROOT, "include", "bastion_cache.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    return {m.group(1): m.group(2).count(",") + 1 for m in re.finditer(r"\b(bastion_\w+)\s*\(([^)]*)\)\s*;", src)}


def test_header_and_binding_agree(b):
    names = _declared()
    assert tuple(names) == b.CACHE_SYMBOLS
    for n, args in names.items():
        assert len(getattr(b.lib(), n).argtypes) == args, n
    for code in (b.STATUS_BAD_PAGE, b.STATUS_BAD_ROW):
        assert b.bastion_status_string(code) != "unknown code"


class _Struct(ctypes.Structure):
    """bastion_paged_cache, as the header declares it."""
    _fields_ = [("k_pool", vp), ("v_pool", vp), ("n_pages", ctypes.c_int64), ("stride_page", ctypes.c_int64),
                ("stride_slot", ctypes.c_int64), ("stride_head", ctypes.c_int64), ("page_table", vp)] + \
               [(n, ctypes.c_int32) for n in ("dtype", "B", "Hkv", "D", "page_size", "max_pages")]


def test_struct_layout(b):
    """The binding packs the struct's bytes itself: the same size and members as a C struct of that declaration."""
    src = open(os.path.join(ROOT, "include", "bastion_cache.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    body = re.search(r"typedef struct \{(.*?)\} bastion_paged_cache;", src, flags=re.S).group(1)
    names = [n.strip(" *") for line in body.split(";") if line.strip() for n in line.strip().split(None, 1)[1].split(",")]
    assert [n.split()[-1].strip("*") for n in names] == [n for n, _ in _Struct._fields_]
    assert b._PAGED_CACHE.size == ctypes.sizeof(_Struct)
    t = _tensors()
    dev, B, Hkv, D, cap, raw = b._cache(t["k"], t["v"], t["table"])
    s = _Struct.from_buffer_copy(raw)
    assert (dev, B, Hkv, D, cap) == (-1, 2, 2, 128, 48)
    assert (s.k_pool, s.v_pool, s.page_table) == tuple(t[n].data_ptr() for n in ("k", "v", "table"))
    assert (s.n_pages, s.stride_page, s.stride_slot, s.stride_head) == (6, 16 * 2 * 128, 2 * 128, 128)
    assert (s.dtype, s.B, s.Hkv, s.D, s.page_size, s.max_pages) == (1, 2, 2, 128, 16, 3)


def _struct(b, **over):
    v = dict(k_pool=0x100000, v_pool=0x200000, n_pages=100, stride_page=16 * 8 * 128, stride_slot=8 * 128,
             stride_head=128, page_table=0x300000, dtype=1, B=4, Hkv=8, D=128, page_size=16, max_pages=20)
    v.update(over)
    return ctypes.byref(_Struct(*(v[n] for n, _ in _Struct._fields_)))


APPEND = dict(k_new=vp(0x400000), v_new=vp(0x500000), n_rows=16, sb=16 * 1024, sr=1024, sh=128, rows=None, m=16,
              n_new=None, seq_len=vp(0x600000), seq_len_out=vp(0x600000), n_seen=vp(0x700000),
              n_seen_out=vp(0x700000), acc=vp(0x800000), pos=vp(0x900000), ws=vp(0xa00000), ws_bytes=1 << 20,
              status=vp(0xb00000), stream=None)
ATTEND = dict(q=vp(0x400000), Hq=32, q_stride_b=32 * 128, seq_len=vp(0x500000), scale=ctypes.c_float(0.1),
              out=vp(0x600000), lse=None, acc=vp(0x10000000), acc_out=vp(0x20000000), ws=vp(0xa00000),
              ws_bytes=1 << 30, status=vp(0xb00000), stream=None)
EVICT = dict(seq_len=vp(0x400000), n_seen=vp(0x500000), acc=vp(0x10000000), pos=vp(0x20000000), budget=64, sink=4,
             recent=16, seq_len_out=vp(0x400000), acc_out=vp(0x10000000), pos_out=vp(0x20000000), ws=vp(0xa00000),
             ws_bytes=1 << 30, status=vp(0xb00000), stream=None)
CALLS = {"append": ("bastion_paged_append", APPEND), "attend": ("bastion_paged_attention", ATTEND),
         "evict": ("bastion_paged_evict", EVICT)}


def _call(b, which, cache=None, **over):
    name, args = CALLS[which]
    assert set(over) <= set(args)
    return getattr(b.lib(), name)(_struct(b, **(cache or {})), *{**args, **over}.values())


CACHE_REFUSALS = [
    (dict(k_pool=None), NULL), (dict(v_pool=None), NULL), (dict(page_table=None), NULL),
    (dict(dtype=0), DTYPE), (dict(dtype=7), DTYPE),
    (dict(B=0), SIZE), (dict(B=1025), SIZE), (dict(Hkv=0), SIZE), (dict(B=1024, Hkv=64), SIZE),
    (dict(n_pages=0), SIZE), (dict(n_pages=1 << 31), SIZE), (dict(max_pages=0), SIZE),
    (dict(max_pages=(1 << 24) + 1), SIZE), (dict(D=0), SIZE), (dict(page_size=0), SIZE),
    (dict(D=96), UNSUPPORTED), (dict(D=256), UNSUPPORTED), (dict(page_size=4), UNSUPPORTED),
    (dict(page_size=24), UNSUPPORTED), (dict(page_size=256), UNSUPPORTED),
    (dict(stride_page=16 * 1024 + 4), SIZE), (dict(stride_slot=64), SIZE), (dict(stride_head=0), SIZE),
    (dict(stride_slot=-1024), SIZE),
    (dict(k_pool=0x100008), ALIGN), (dict(v_pool=0x200002), ALIGN),
]


@pytest.mark.parametrize("which", list(CALLS))
@pytest.mark.parametrize("over,code", CACHE_REFUSALS)
def test_cache_refusals(b, which, over, code):
    assert _call(b, which, over) == code


@pytest.mark.parametrize("which,over,code", [
    ("append", dict(k_new=None), NULL), ("append", dict(seq_len=None), NULL), ("append", dict(status=None), NULL),
    ("append", dict(ws=None), NULL), ("append", dict(acc=None), NULL), ("append", dict(pos=None), NULL),
    ("append", dict(n_seen=None), NULL), ("append", dict(n_seen=None, n_seen_out=None), NULL),
    ("append", dict(m=0), SIZE), ("append", dict(m=17), SIZE), ("append", dict(n_rows=0), SIZE),
    ("append", dict(rows=vp(0xc00000), m=1025), SIZE), ("append", dict(sr=1028), SIZE), ("append", dict(sh=-128), SIZE),
    ("append", dict(k_new=vp(0x400008)), ALIGN), ("append", dict(ws=vp(0xa00010)), ALIGN),
    ("append", dict(ws_bytes=16), WORKSPACE), ("append", dict(seq_len_out=vp(0x600004)), UNSUPPORTED),
    ("append", dict(n_seen_out=vp(0x6ffffc)), UNSUPPORTED),
    ("attend", dict(q=None), NULL), ("attend", dict(out=None), NULL), ("attend", dict(acc=None), NULL),
    ("attend", dict(acc_out=None), NULL), ("attend", dict(Hq=33), SIZE), ("attend", dict(Hq=0), SIZE),
    ("attend", dict(Hq=136), UNSUPPORTED), ("attend", dict(scale=ctypes.c_float(0.0)), SIZE),
    ("attend", dict(scale=ctypes.c_float(float("nan"))), SIZE), ("attend", dict(scale=ctypes.c_float(float("inf"))), SIZE),
    ("attend", dict(q_stride_b=4100), SIZE), ("attend", dict(q=vp(0x400008)), ALIGN),
    ("attend", dict(out=vp(0x600008)), ALIGN), ("attend", dict(ws_bytes=1024), WORKSPACE),
    ("attend", dict(acc_out=vp(0x10000040)), UNSUPPORTED),
    ("evict", dict(acc=None), NULL), ("evict", dict(pos_out=None), NULL), ("evict", dict(n_seen=None), NULL),
    ("evict", dict(budget=0), SIZE), ("evict", dict(sink=-1), SIZE), ("evict", dict(recent=-1), SIZE),
    ("evict", dict(sink=40, recent=25), SIZE), ("evict", dict(ws_bytes=64), WORKSPACE),
    ("evict", dict(acc_out=vp(0x10000010)), UNSUPPORTED), ("evict", dict(acc=vp(0x10000004)), ALIGN),
    ("evict", dict(pos_out=vp(0x20000008)), ALIGN), ("attend", dict(acc=vp(0x10000008)), ALIGN), ("evict", dict(pos_out=vp(0x1fffff00)), UNSUPPORTED),
    ("evict", dict(ws=vp(0xa00080)), ALIGN), ("evict", dict(n_seen=vp(0x400000)), UNSUPPORTED),
])
def test_call_refusals(b, which, over, code):
    assert _call(b, which, **over) == code


@pytest.mark.parametrize("over", [
    dict(seq_len_out=vp(0x700004)), dict(n_seen_out=vp(0x600008)), dict(n_new=vp(0x600004)), dict(n_new=vp(0x6ffffc)),
    dict(seq_len_out=vp(0xd00000), n_seen_out=vp(0xd00000)), dict(seq_len_out=vp(0xd00000), n_seen_out=vp(0xd00004)),
])
def test_lengths_over_part_of_one_another(b, over):
    """A request's last CTA writes its lengths while others may still read their own requests' entries."""
    assert _call(b, "append", **over) == UNSUPPORTED


@pytest.mark.parametrize("over", [
    dict(out=vp(0x400010)), dict(out=vp(0x3ffff0)), dict(q_stride_b=33 * 128, out=vp(0x400000)),
    dict(q_stride_b=64 * 128, out=vp(0x400000 + 64 * 128 * 2 * 3 + 32 * 128 * 2 - 16)),
])
def test_outputs_over_part_of_the_queries(b, over):
    """out is q's own memory, row for row, or none of it."""
    assert _call(b, "attend", **over) == UNSUPPORTED


def test_workspace_queries(b):
    assert b.bastion_paged_append_workspace_bytes(4) > 0
    assert b.bastion_paged_append_workspace_bytes(0) == 0 == b.bastion_paged_append_workspace_bytes(1025)
    w = b.bastion_paged_attention_workspace_bytes
    assert 0 < w(4, 32, 8, 128, 4096, False) < w(4, 32, 8, 128, 4096, True)
    assert w(4, 33, 8, 128, 4096, False) == w(4, 32, 8, 96, 4096, False) == w(4, 32, 1, 128, 4096, False) == 0
    assert w(4, 32, 8, 128, (1 << 28) + 1, False) == 0
    assert b.bastion_paged_evict_workspace_bytes(4, 8, 4096) > 0
    assert b.bastion_paged_evict_workspace_bytes(1024, 64, 4096) == 0


def _tensors(B=2, Hq=8, Hkv=2, D=128, page=16, pages=6, max_pages=3):
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    return dict(k=bf(pages, page, Hkv, D), v=bf(pages, page, Hkv, D), table=i32(B, max_pages), lens=i32(B), st=i32(B),
                q=bf(B, Hq, D), out=bf(B, Hq, D), acc=torch.zeros(B, Hkv, max_pages * page),
                pos=i32(B, Hkv, max_pages * page), new=bf(B, 4, Hkv, D), ws=torch.zeros(1 << 20, dtype=torch.uint8))


def _attend(b, t, **kw):
    b.bastion_paged_attention(t["q"], t["k"], t["v"], t["table"], t["lens"], 0.1, t["out"], t["ws"], t["st"], **kw)


@pytest.mark.parametrize("change,match", [
    (lambda t: t.update(k=t["k"].float()), "one shape and dtype"),
    (lambda t: t.update(k=t["k"].float(), v=t["v"].float()), "bfloat16 or float16"),
    (lambda t: t.update(k=t["k"][:5]), "one shape"),
    (lambda t: t.update(v=t["v"].transpose(1, 2).contiguous().transpose(1, 2)), "equal strides"),
    (lambda t: t.update(k=t["k"][0], v=t["v"][0]), "n_pages"),
    (lambda t: t.update(table=t["table"].long()), "page_table"),
    (lambda t: t.update(table=t["table"][0]), "page_table"),
    (lambda t: t.update(q=t["q"].half()), "pools' dtype"),
    (lambda t: t.update(q=t["q"][:, :, :64]), "q must be"),
    (lambda t: t.update(q=t["q"].transpose(0, 1).contiguous().transpose(0, 1)), "heads of q"),
    (lambda t: t.update(out=t["out"].float()), "out"),
    (lambda t: t.update(lens=t["lens"].long()), "seq_len"),
    (lambda t: t.update(st=t["st"][:1]), "status"),
    (lambda t: t.update(ws=t["ws"].int()), "workspace"),
    (lambda t: None, "CUDA device"),
])
def test_binding_refuses_attention_arguments(b, change, match):
    t = _tensors()
    change(t)
    with pytest.raises(b.BastionError, match=match):
        _attend(b, t)


def test_marshal_declines_what_the_binding_refuses(b):
    """The compiled short way takes only calls that are right (CUDA tensors): for anything else it calls nothing,
    raises nothing and leaves the binding's own checks to speak."""
    m, t = b._marshal, _tensors()
    assert m is not None
    att = [t["q"], t["k"], t["v"], t["table"], t["lens"], 0.1, t["out"], t["ws"], t["st"], None, None, None, None]
    app = [t["new"], t["new"], t["k"], t["v"], t["table"], t["lens"], t["lens"], t["ws"], t["st"]] + [None] * 7
    ev = [t["k"], t["v"], t["table"], t["lens"], t["lens"], t["acc"], t["pos"], 8, 0, 0, t["lens"], t["acc"], t["pos"],
          t["ws"], t["st"], None]
    for f, args in ((m.attention, att), (m.append, app), (m.evict, ev)):
        assert f(*args) is None            # CPU tensors
        assert f() is None and f(*args, None) is None
        for i in range(len(args)):
            for bad in (None, 3, "x", 1 << 70, torch.zeros(1, 1, 1, 1, 1), object()):
                assert f(*args[:i], bad, *args[i + 1:]) is None


def test_strides_of_single_entries_do_not_matter(b):
    """One token's rows [B, 1, Hkv, D], transposed or not: the same memory, whatever the stride of the 1 says."""
    t = _tensors()
    one = torch.zeros(2, 1, 2, 128, dtype=torch.bfloat16)
    other = torch.zeros(2, 2, 1, 128, dtype=torch.bfloat16).transpose(1, 2)
    assert one.stride() != other.stride()
    with pytest.raises(b.BastionError, match="CUDA device"):  # and nothing else
        b.bastion_paged_append(one, other, t["k"], t["v"], t["table"], t["lens"], t["lens"], t["ws"], t["st"])
    k = t["k"][:1]
    v = torch.as_strided(k, k.shape, (8, *k.stride()[1:]))
    assert v.stride() != k.stride()
    with pytest.raises(b.BastionError, match="CUDA device"):
        b.bastion_paged_append(one, one, k, v, t["table"], t["lens"], t["lens"], t["ws"], t["st"])


class _Fake:
    """What the short way looks at of a tensor; on device 0."""

    def __init__(self, t):
        self.t, self.dtype, self.shape = t, t.dtype, tuple(t.shape)
        self.stride, self.is_contiguous, self.data_ptr = t.stride, t.is_contiguous, t.data_ptr

    def get_device(self):
        return 0


def test_marshal_calls_without_the_interpreters_lock(b):
    """A function that says whether its thread holds the lock, in place of the library's three."""
    m, t = b._marshal, {n: _Fake(x) for n, x in _tensors().items()}
    held = ctypes.cast(ctypes.pythonapi.PyGILState_Check, vp).value
    try:
        m.init(torch.bfloat16, torch.float16, torch.float32, torch.int32, torch.uint8, lambda: 0, lambda dev: 0, held,
               held, held)
        assert m.attention(t["q"], t["k"], t["v"], t["table"], t["lens"], 0.1, t["out"], t["ws"], t["st"], None, None,
                           None, None) == 0
        assert m.append(t["new"], t["new"], t["k"], t["v"], t["table"], t["lens"], t["lens"], t["ws"], t["st"],
                        *[None] * 7) == 0
        assert m.evict(t["k"], t["v"], t["table"], t["lens"], t["lens"], t["acc"], t["pos"], 8, 0, 0, t["lens"],
                       t["acc"], t["pos"], t["ws"], t["st"], None) == 0
    finally:
        b._marshal = b._load_marshal(b.lib())


def test_binding_refuses_other_arguments(b):
    t = _tensors()
    with pytest.raises(b.BastionError, match="lse"):
        _attend(b, t, lse=torch.zeros(2, 8, dtype=torch.float64))
    with pytest.raises(b.BastionError, match="acc"):
        _attend(b, t, acc=t["acc"][:, :, :40], acc_out=t["acc"])

    def append(k=t["new"], v=t["new"], **kw):
        b.bastion_paged_append(k, v, t["k"], t["v"], t["table"], t["lens"], t["lens"], t["ws"], t["st"], **kw)

    with pytest.raises(b.BastionError, match="pools' dtype"):
        append(k=t["new"].half())
    with pytest.raises(b.BastionError, match="pools' dtype"):
        append(k=t["new"][:, :, :1], v=t["new"][:, :, :1])
    with pytest.raises(b.BastionError, match="equal strides"):
        append(v=t["new"].transpose(1, 2).contiguous().transpose(1, 2))
    with pytest.raises(b.BastionError, match="rows"):
        append(rows=torch.zeros(2, 4, dtype=torch.int64))
    with pytest.raises(b.BastionError, match="rows"):
        append(rows=torch.zeros(8, dtype=torch.int32))
    with pytest.raises(b.BastionError, match="n_new"):
        append(n_new=torch.zeros(3, dtype=torch.int32))
    with pytest.raises(b.BastionError, match="pos"):
        append(acc=t["acc"], pos=t["pos"].long())
    with pytest.raises(b.BastionError, match="CUDA device"):
        append()

    def evict(**kw):
        a = dict(seq_len=t["lens"], n_seen=t["lens"], acc=t["acc"], pos=t["pos"], budget=8)
        a.update(kw)
        b.bastion_paged_evict(t["k"], t["v"], t["table"], a["seq_len"], a["n_seen"], a["acc"], a["pos"], a["budget"], 0, 0,
                              t["lens"], t["acc"], t["pos"], t["ws"], t["st"])

    with pytest.raises(b.BastionError, match="n_seen"):
        evict(n_seen=t["lens"].long())
    with pytest.raises(b.BastionError, match="acc"):
        evict(acc=t["acc"].double())
    with pytest.raises(b.BastionError, match="32 bits"):
        evict(budget=(1 << 32) + 8)
    with pytest.raises(b.BastionError, match="CUDA device"):
        evict()
    with pytest.raises(b.BastionError, match="n_pages"):
        b.PagedCache(1, 1, 1, 64, 8, 1, "cpu", page_table=torch.zeros(1, 1, dtype=torch.int32))
