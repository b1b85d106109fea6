"""Page numbers that are none, on their way back to the free list."""
import pytest
import torch

from gpuhelp import dev
from test_gpu_plan import Plan

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad", [-1, -2 ** 31, 2 ** 31 - 1, None])
@pytest.mark.parametrize("taken", [False, True])
def test_a_page_that_is_none_is_given_back(cuda_lib, bad, taken):
    """The request that held it is told, whether the number stays on the list or another request takes it at once, which is
    told as well; the others are served as ever."""
    # request 1 has ended and holds four pages; request 2 grows by three where `taken`, which are the last that came back
    p = Plan([5, 0, 20, 7], 64, 16, [1, 0, 44 if taken else 1, 1], False, None, True, 6, [1, 4, 2, 1], 8)
    at = p.table[1][3]
    p.t["table"][1, 3] = p.n_pages if bad is None else bad
    p.run()
    torch.cuda.synchronize()
    assert p.status.tolist() == [0, 64, 64 if taken else 0, 0]
    given = [x for x in p.table[1][:3]]
    number = p.n_pages if bad is None else bad
    assert p.t["held_out"].tolist() == [1, 0, 4 if taken else 2, 1] and at not in p.t["table"].tolist()[2]
    stack, left = p.t["stack"].tolist(), int(p.t["n_free_out"])
    assert stack[:6] == p.stack[:6]
    if taken:
        assert left == 8 and stack[6:8] == given[:2] and p.t["table"].tolist()[2][2:4] == [number, given[2]]
        slots = p.slots.tolist()[2 * 64:2 * 64 + 44]
        assert slots[:12] == [p.table[2][1] * 16 + i for i in range(4, 16)] and slots[12:28] == [-1] * 16
        assert slots[28:] == [given[2] * 16 + i for i in range(16)]
    else:
        assert left == 10 and stack[6:10] == given + [number]


def test_pages_kept_are_not_looked_at(cuda_lib):
    """Without trim nothing comes back, and entries that no row uses are not read."""
    p = Plan([5, 0], 8, 16, [1, 0], False, None, False, 6, [1, 4], 8)
    p.t["table"][1, 3] = -7
    p.run()
    torch.cuda.synchronize()
    assert p.status.tolist() == [0, 0] and p.t["held_out"].tolist() == [1, 4]
