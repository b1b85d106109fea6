"""Arrays of the paged cache's calls that lie over one another: refused by the C ABI's host checks (fake pointers, never
dereferenced).  A call whose arrays are apart gets as far as the last check, the workspace's size."""
import ctypes

import pytest

from test_paged_refusals import UNSUPPORTED, WORKSPACE, _call, b  # noqa: F401

vp = ctypes.c_void_p
B, SLOTS = 4, 4 * 8 * 20 * 16 * 4  # requests; bytes of acc and of pos


def _is(b, which, over, code):  # noqa: F811
    """Refused for the overlap before the workspace is looked at, or for the workspace alone."""
    assert _call(b, which, ws_bytes=0, **over) == code


ROWS = dict(rows=vp(0xc00000), m=17)  # B * 17 entries


@pytest.mark.parametrize("over", [
    dict(ROWS, seq_len=vp(0xd00000), seq_len_out=vp(0xc00000)), dict(ROWS, seq_len=vp(0xd00000), seq_len_out=vp(0xc00000 + B * 17 * 4 - 4)),
    dict(ROWS, n_seen=vp(0xd00000), n_seen_out=vp(0xc00040)), dict(ROWS, rows=vp(0x600008)),  # in place, the list over it
    dict(seq_len_out=vp(0x300000)), dict(n_seen_out=vp(0x300000 + 4 * 20 * 4 - 4)),      # the page table
    dict(seq_len_out=vp(0x800000)), dict(seq_len_out=vp(0x900000 + SLOTS - 4)), dict(seq_len_out=vp(0xb00000)),
    dict(ROWS, rows=vp(0x800000 + SLOTS - 16)), dict(pos=vp(0x800000)), dict(pos=vp(0x800000 + SLOTS - 16)),
    dict(acc=vp(0x600000)), dict(pos=vp(0x300000)), dict(status=vp(0x900000)), dict(status=vp(0x600000)),
    dict(n_new=vp(0x800010)), dict(n_new=vp(0xb00000)),
])
def test_append(b, over):  # noqa: F811
    _is(b, "append", over, UNSUPPORTED)


@pytest.mark.parametrize("over", [
    dict(), ROWS, dict(ROWS, rows=vp(0x600000 + B * 4)), dict(ROWS, rows=vp(0x600000 - B * 17 * 4)),
    dict(seq_len_out=vp(0x800000 - B * 4)), dict(seq_len_out=vp(0x800000 + SLOTS)), dict(pos=vp(0x800000 + SLOTS)),
    dict(acc=None, pos=None, n_seen=None, n_seen_out=None), dict(n_new=vp(0xd00000)), dict(n_new=vp(0x600000)),
    dict(n_seen=vp(0x600000), n_seen_out=vp(0x600000)),
])
def test_append_apart(b, over):  # noqa: F811
    _is(b, "append", over, WORKSPACE)


A0, P0, L0 = 0x10000000, 0x20000000, 0x400000  # evict's acc, pos and seq_len, each in place


@pytest.mark.parametrize("over", [
    dict(acc_out=vp(P0)), dict(pos_out=vp(A0)), dict(acc_out=vp(P0 + SLOTS - 16)), dict(pos_out=vp(A0 - SLOTS + 16)),
    dict(acc_out=vp(0x30000000), pos_out=vp(0x30000000)), dict(acc_out=vp(0x30000000), pos_out=vp(0x30000000 + SLOTS - 16)),
    dict(pos=vp(A0), pos_out=vp(P0)),  # acc in place over pos
    dict(seq_len_out=vp(A0)), dict(seq_len_out=vp(P0 + SLOTS - 4)), dict(seq_len_out=vp(0x300000)),
    dict(seq_len_out=vp(0xb00000)), dict(acc_out=vp(L0)), dict(pos_out=vp(0x500000)), dict(acc_out=vp(0x300000)),
    dict(status=vp(L0)), dict(status=vp(0x500000)), dict(status=vp(A0)), dict(status=vp(P0 + 4)),
    dict(acc_out=vp(0x30000000), seq_len_out=vp(0x30000000)), dict(status=vp(0x300000)),
])
def test_evict(b, over):  # noqa: F811
    _is(b, "evict", over, UNSUPPORTED)


@pytest.mark.parametrize("over", [
    dict(), dict(acc_out=vp(A0 + SLOTS), pos_out=vp(P0 + SLOTS), seq_len_out=vp(L0 + B * 4)),
    dict(pos=vp(A0 + SLOTS), pos_out=vp(A0 + SLOTS)), dict(acc_out=vp(P0 - SLOTS)), dict(acc=vp(P0), acc_out=vp(A0)) | dict(pos=vp(P0 + SLOTS), pos_out=vp(P0 + SLOTS)),
    dict(seq_len_out=vp(0x500000 + B * 4)),
])
def test_evict_apart(b, over):  # noqa: F811
    _is(b, "evict", over, WORKSPACE)


Q0, Q, O0, W0, WO = 0x400000, 32 * 128 * 2, 0x600000, 0x10000000, 0x20000000  # q, a row of it, out, acc, acc_out
WIDE = dict(q_stride_b=2 * 32 * 128)  # rows of a fused projection: gaps as wide as they are
LSE = B * 32 * 4


@pytest.mark.parametrize("over", [
    dict(lse=vp(0x500000)), dict(lse=vp(0x300000)), dict(lse=vp(O0)), dict(lse=vp(O0 + B * Q - 4)), dict(lse=vp(W0)),
    dict(lse=vp(WO + SLOTS - 4)), dict(lse=vp(0xb00000)), dict(lse=vp(Q0)), dict(lse=vp(Q0 + B * Q - 4)),
    dict(lse=vp(Q0 - LSE + 4)), dict(WIDE, lse=vp(Q0 + 2 * Q - 4)), dict(WIDE, lse=vp(Q0 + 2 * Q - LSE + 4)),
    dict(WIDE, lse=vp(Q0 + 6 * Q)), dict(WIDE, status=vp(Q0 + 7 * Q - 4)), dict(q_stride_b=0, lse=vp(Q0 + Q - 4)),
    dict(out=vp(0x500000)), dict(out=vp(0x300000)), dict(out=vp(W0)), dict(out=vp(WO + SLOTS - 16)), dict(out=vp(0xb00000)),
    dict(acc_out=vp(0x500000)), dict(acc_out=vp(0x300000)), dict(acc_out=vp(Q0)), dict(WIDE, acc_out=vp(Q0 + Q)),
    dict(status=vp(0x500000)), dict(status=vp(0x300000)), dict(status=vp(W0)), dict(status=vp(O0)),
])
def test_attention(b, over):  # noqa: F811
    _is(b, "attend", over, UNSUPPORTED)


@pytest.mark.parametrize("over", [
    dict(), dict(lse=vp(O0 + B * Q)), dict(lse=vp(O0 - LSE)), dict(lse=vp(Q0 + B * Q)), dict(lse=vp(Q0 - LSE)),
    dict(WIDE, lse=vp(Q0 + Q)), dict(WIDE, lse=vp(Q0 + 2 * Q - LSE)), dict(WIDE, lse=vp(Q0 + 7 * Q)),
    dict(WIDE, status=vp(Q0 + 5 * Q)), dict(q_stride_b=0, lse=vp(Q0 + Q)), dict(q_stride_b=0, lse=vp(Q0 - LSE)),
    dict(out=vp(Q0)), dict(acc_out=vp(W0)), dict(acc=None, acc_out=None, lse=vp(WO)), dict(acc_out=vp(W0 + SLOTS)),
])
def test_attention_apart(b, over):  # noqa: F811
    _is(b, "attend", over, WORKSPACE)
