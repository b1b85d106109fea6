"""GPU parity of the page plan with a sequential reference: every number exactly."""
import pytest
import torch

import layerref as ref
from gpuhelp import dev

pytestmark = pytest.mark.gpu


class Plan:
    """One call's tensors.  lens: used slots; held: pages (None: as many as lens needs, and one more here and there)."""

    def __init__(self, lens, m, page=16, n_new=None, packed=False, n_rows=None, trim=False, spare=None, held=None,
                 max_pages=None, seed=0, inplace=False, n_pages=None):
        from draft_tree_build_gb300 import bastion
        self.b = bastion
        g = torch.Generator().manual_seed(seed)
        B = len(lens)
        need = [-(-max(0, n) // page) for n in lens]
        self.max_pages = max_pages or max(1, max(-(-(max(0, n) + m) // page) for n in lens) + 1)
        if held is None:
            held = [min(self.max_pages, k + int(torch.randint(0, 3, (1,), generator=g)) // 2) for k in need]
        used = sum(max(0, min(h, self.max_pages)) for h in held)
        if spare is None:
            spare = sum(-(-(max(0, n) + m) // page) for n in lens) + 5
        self.n_pages = n_pages or used + spare + 7
        ids = torch.randperm(self.n_pages, generator=g).tolist()
        self.table = [[2 ** 31 - 1 if i % 2 else -5] * self.max_pages for i in range(B)]
        at = 0
        for r in range(B):
            k = max(0, min(held[r], self.max_pages))
            self.table[r][:k] = ids[at:at + k]
            at += k
        self.stack = ids[at:at + spare] + [-9] * (self.n_pages - spare)
        self.args = dict(page=page, n_pages=self.n_pages, lens=list(lens), m=m, held=held, n_free=spare, packed=packed,
                         n_rows=n_rows if packed else B * m, n_new=n_new, trim=trim)
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev())  # noqa: E731
        self.t = dict(table=i32(self.table), lens=i32(lens), held=i32(held), stack=i32(self.stack), n_free=i32([spare]),
                      n_new=None if n_new is None else i32(n_new))
        self.t["lens_out"] = self.t["lens"] if inplace else i32([7] * B)
        self.t["held_out"] = self.t["held"] if inplace else i32([7] * B)
        self.t["n_free_out"] = self.t["n_free"] if inplace else i32([7])
        rows = self.args["n_rows"]
        self.slots = torch.full((rows,), 77, dtype=torch.int64, device=dev())
        self.pos = torch.full((rows,), 77, dtype=torch.int32, device=dev())
        self.start = i32([7] * (B + 1)) if packed else None
        self.status = i32([0] * B)
        self.ws = bastion.workspace(bastion.bastion_paged_plan_workspace_bytes(B), dev())

    def run(self, stream=None):
        t = self.t
        self.b.bastion_paged_plan(t["table"], self.args["page"], t["lens"], self.args["m"], t["held"], t["held_out"],
                                  t["stack"], t["n_free"], t["n_free_out"], self.slots, self.pos, self.ws, self.status,
                                  n_new=t["n_new"], row_start=self.start, seq_len_out=t["lens_out"],
                                  trim=self.args["trim"], stream=stream)
        return self

    def check(self):
        torch.cuda.synchronize()
        want = ref.plan(self.table, stack=self.stack, **self.args)
        got = dict(table=self.t["table"], held=self.t["held_out"], stack=self.t["stack"], n_free=self.t["n_free_out"],
                   slots=self.slots, pos=self.pos, lens=self.t["lens_out"], status=self.status)
        if self.start is not None:
            got["start"] = self.start
        for name, x in got.items():
            w = want[name] if name != "n_free" else [want[name]]
            assert x.tolist() == w, name
        assert not bool(self.ws.any())
        return want


EDGES = [0, 1, 15, 16, 17, 31, 32, 33, 127, 128, 129, 500, 0]


@pytest.mark.parametrize("page", [8, 16, 32, 64, 128])
@pytest.mark.parametrize("m", [1, 2, 17, 128, 500])
@pytest.mark.parametrize("packed", [False, True])
def test_lengths_at_every_edge(cuda_lib, page, m, packed):
    Plan(EDGES, m, page, packed=packed, n_rows=len(EDGES) * m + 3, seed=m).run().check()


@pytest.mark.parametrize("B", [1, 2, 31, 255, 256, 257, 700, 1024])
@pytest.mark.parametrize("packed,trim,inplace", [(False, True, False), (True, False, True), (True, True, True)])
def test_batches(cuda_lib, B, packed, trim, inplace):
    g = torch.Generator().manual_seed(B)
    lens = torch.randint(0, 300, (B,), generator=g).tolist()
    new = torch.randint(-2, 50, (B,), generator=g).tolist()
    for r in range(0, B, 5):
        lens[r], new[r] = 0, 0
    held = [-(-n // 16) + (3 if r % 5 == 0 else r % 2) for r, n in enumerate(lens)]
    Plan(lens, 40, 16, new, packed, 40 * B, trim, held=held, seed=B, inplace=inplace, max_pages=25).run().check()


@pytest.mark.parametrize("spare", [0, 1, 2, 7, 20, 33])
@pytest.mark.parametrize("trim", [False, True])
@pytest.mark.parametrize("packed", [False, True])
def test_too_few_pages(cuda_lib, spare, trim, packed):
    """The first request that finds too few, and all after it that need some, get nothing; the others go on."""
    lens = [5, 100, 16, 0, 31, 64, 7, 48, 200, 0]
    new = [20, 1, 1, 64, 1, 0, 60, 2, 0, 1]
    held = [1, 9, 1, 0, 2, 6, 1, 3, 15, 0]
    p = Plan(lens, 64, 16, new, packed, 300, trim, spare, held, 20, seed=spare)
    want = p.run().check()
    # 12 pages are asked for; the second, sixth and ninth requests hold two too many each
    assert (ref.NO_PAGE in want["status"]) == (spare + 6 * trim < 12)


@pytest.mark.parametrize("rows", [1, 5, 64, 99, 100, 101, 1000])
def test_too_few_packed_rows(cuda_lib, rows):
    p = Plan([10] * 8, 40, 8, [30, 0, 30, 40, 1, 0, 7, 3], True, rows, True, max_pages=9)
    want = p.run().check()
    assert want["start"][-1] <= rows and (ref.OVERFLOW in want["status"]) == (rows < 111)


def test_status(cuda_lib):
    """Lengths and counts of pages that cannot be: the request keeps what it has, the others are served."""
    lens = [-1, 10, 200, 161, 20, 40, 3, -2 ** 31, 2 ** 31 - 1]
    held = [2, 0, 10, 10, -1, 11, 1, 0, 0]
    for packed in (False, True):
        want = Plan(lens, 8, 16, None, packed, 72, True, 20, held, 10).run().check()
        assert want["status"] == [8, 64, 8, 8, 64, 64, 0, 8, 8]


def test_pages_that_are_none(cuda_lib):
    """Entries of the free list and the table that are no pages of the pool: no slots there."""
    p = Plan([20, 3], 30, 16, None, False, None, False, 8, [2, 1], 8)
    p.t["table"][0, 1] = p.n_pages
    p.t["stack"][7] = -3  # the first page taken: request 0's third
    p.run()
    torch.cuda.synchronize()
    assert p.status.tolist() == [64, 0]
    slots, pos = p.slots.tolist(), p.pos.tolist()
    assert pos[:30] == list(range(20, 50)) and slots[:28] == [-1] * 28 and min(slots[28:30]) >= 0
    assert min(slots[30:]) >= 0
    for high in (False, True):  # a free list that cannot be
        q = Plan([3], 1, 16, held=[1], max_pages=2)
        left = q.n_pages if high else 0
        q.t["n_free"][0] = q.n_pages + 5 if high else -4
        q.run()
        torch.cuda.synchronize()
        assert q.status.tolist() == [64] and q.t["n_free_out"].tolist() == [left]


def test_a_captured_plan_feeds_itself(cuda_lib):
    """A decoding loop of one captured call, everything in place: lengths, pages and the free list go on."""
    p = Plan([0, 5, 16, 100], 3, 8, [1, 2, 3, 1], False, trim=True, spare=40, max_pages=30, inplace=True)
    g = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.graph(g, stream=side):
        p.run()
    for _ in range(20):
        g.replay()
        want = p.check()
        p.table, p.stack = want["table"], want["stack"]
        p.args.update(lens=want["lens"], held=want["held"], n_free=want["n_free"])


def test_long_prompts_and_odd_views(cuda_lib):
    """More rows than a grid's first pass; outputs that are only 8- and 4-byte aligned."""
    lens = [1000 * i for i in range(16)]
    p = Plan(lens, 60000, 64, None, True, 16 * 60000 + 5, max_pages=2000)
    slots, pos = torch.zeros(16 * 60000 + 6, dtype=torch.int64, device=dev()), torch.zeros(16 * 60000 + 6, dtype=torch.int32, device=dev())
    p.slots, p.pos = slots[1:], pos[1:]
    p.run().check()
    assert int(slots[0]) == 0 and int(pos[0]) == 0


def test_two_streams(cuda_lib):
    a, b = Plan(EDGES, 17), Plan([900] * 9, 40, 8)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(10):
        a.run(s1)
        b.run(s2)
    a.check()
    b.check()
