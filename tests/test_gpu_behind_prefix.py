"""Positions of tokens behind a shared prefix: planned, turned, stored and attended to, they are those of one sequence."""
import pytest
import torch

import layerref as ref
import pagedref
from gpuhelp import dev
from test_gpu_plan import EDGES, Plan

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=dev())


class Offset(Plan):
    def __init__(self, offset, *args, **kw):
        super().__init__(*args, **kw)
        self.offset = i32(offset)

    def run(self, stream=None):
        t = self.t
        self.b.bastion_paged_plan(t["table"], self.args["page"], t["lens"], self.args["m"], t["held"], t["held_out"],
                                  t["stack"], t["n_free"], t["n_free_out"], self.slots, self.pos, self.ws, self.status,
                                  n_new=t["n_new"], row_start=self.start, seq_len_out=t["lens_out"],
                                  trim=self.args["trim"], stream=stream, pos_offset=self.offset)
        return self

    def check(self):
        """The plain plan's numbers, the positions moved; rows without a token keep their -1."""
        torch.cuda.synchronize()
        want = ref.plan(self.table, stack=self.stack, **self.args)
        B, m = len(self.args["lens"]), self.args["m"]
        who = [r for r in range(B) for _ in range(want["start"][r + 1] - want["start"][r])] if self.start is not None else \
            [r for r in range(B) for _ in range(m)]
        offset = self.offset.tolist()
        moved = [p + offset[r] if p >= 0 else p for p, r in zip(want["pos"], who)] + [-1] * (len(want["pos"]) - len(who))
        assert self.pos.tolist() == moved and self.slots.tolist() == want["slots"]
        assert self.status.tolist() == want["status"] and self.t["table"].tolist() == want["table"]
        assert self.t["lens_out"].tolist() == want["lens"] and self.t["held_out"].tolist() == want["held"]


@pytest.mark.parametrize("m", [1, 17, 128])
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("marshal", [True, False])
def test_plans(cuda_lib, monkeypatch, m, packed, marshal):
    if not marshal:
        monkeypatch.setattr(cuda_lib, "_marshal", None)
    offset = [(1 << 20) * i + 7 * i for i in range(len(EDGES))]
    Offset(offset, EDGES, m, 16, packed=packed, n_rows=len(EDGES) * m + 3, seed=m).run().check()


def test_offsets_at_their_ends(cuda_lib):
    """The last that leaves room for the capacity, and those past it: the request is told and gets nothing."""
    cap = 10 * 16
    top = 2 ** 31 - 1 - cap
    p = Offset([0, top, top + 1, -1, 2 ** 31 - 1, -2 ** 31, 5], [100] * 7, 20, 16, [20, 60, 20, 20, 20, 0, 20], max_pages=10)
    p.run()
    torch.cuda.synchronize()
    assert p.status.tolist() == [0, 0, 8, 8, 8, 8, 0]
    pos = p.pos.view(7, 20).tolist()
    assert pos[0] == list(range(100, 120)) and pos[6] == list(range(105, 125)) and pos[1][0] == top + 100
    assert pos[1][19] == top + 119 and all(x == [-1] * 20 for x in pos[2:6])
    assert p.t["lens_out"].tolist() == [120, 120, 100, 100, 100, 100, 120]


def test_many_requests_and_a_long_plan(cuda_lib):
    g = torch.Generator().manual_seed(2)
    lens = torch.randint(0, 300, (1024,), generator=g).tolist()
    offset = torch.randint(0, 1 << 30, (1024,), generator=g).tolist()
    new = torch.randint(-1, 60, (1024,), generator=g).tolist()
    Offset(offset, lens, 50, 8, new, True, 40 * 1024, True, seed=3, inplace=True, max_pages=60).run().check()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("graph", [False, True])
def test_decoding_behind_prefixes_is_decoding_of_one_sequence(cuda_lib, dtype, graph):
    """Two prompts shared by six requests, a seventh without; each request's tokens again, prompt and all, in a cache of its
    own.  Keys have to be the same bits, and the outputs those of the whole sequences in 64 bits."""
    b = cuda_lib
    g = torch.Generator().manual_seed(11)
    B, Hq, Hkv, D, page, steps = 7, 8, 2, 128, 16, 12
    plens, start, first = [200, 77], [0, 4, 6], [30, 1, 16, 0, 45, 17, 60]
    group = [0, 0, 0, 0, 1, 1, None]
    pre = [-(-n // page) for n in plens]
    c = b.PagedCache(B, Hq, Hkv, D, page, 8, dev(), dtype, n_pages=70, new_tokens=60, reserved=sum(pre), prefixes=2)
    whole = b.PagedCache(B, Hq, Hkv, D, page, 24, dev(), dtype, new_tokens=300)
    table = torch.zeros(2, max(pre), dtype=torch.int32)
    table[0, :pre[0]], table[1, :pre[1]] = torch.arange(pre[0]), torch.arange(pre[0], sum(pre))
    tables, lens, starts = table.to(dev()), i32(plens), i32(start)
    offset = i32([plens[x] if x is not None else 0 for x in group])
    freq, factor = b.rope_frequencies(D, 1e6, dev(), "yarn", 4.0)
    weights = [torch.randn(D, generator=g).to(dtype).to(dev()) for _ in range(2)]
    make = lambda n: torch.randn(n, Hq + 2 * Hkv, D, generator=g).to(dtype).to(dev())  # noqa: E731
    cut = lambda x: (x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:])  # noqa: E731
    prompts, own = [make(n) for n in plens], [make(n) for n in first]

    def write(cache, x, pos, slots, out):
        cache.write(*cut(x), pos, slots, freq, out, *weights, factor=factor)

    # the prompts, into the pages set aside for them, by their own positions
    for i, n in enumerate(plens):
        at = torch.arange(n)
        slots = (table[i][at // page] * page + at % page).long().to(dev())
        write(c, prompts[i], at.to(torch.int32).to(dev()), slots, torch.empty(n, Hq, D, dtype=dtype, device=dev()))
    # the requests' first tokens: behind their prompts, and with them
    x = torch.zeros(B * 60, Hq + 2 * Hkv, D, dtype=dtype, device=dev())
    for r in range(B):
        x[60 * r:60 * r + first[r]] = own[r]
    slots, pos = c.reserve(60, i32(first), pos_offset=offset)
    write(c, x, pos, slots, torch.empty(B * 60, Hq, D, dtype=dtype, device=dev()))
    seqs = [torch.cat([prompts[group[r]], own[r]]) if group[r] is not None else own[r] for r in range(B)]
    x = torch.zeros(B * 300, Hq + 2 * Hkv, D, dtype=dtype, device=dev())
    for r in range(B):
        x[300 * r:300 * r + len(seqs[r])] = seqs[r]
    slots, pos = whole.reserve(300, i32([len(s) for s in seqs]))
    write(whole, x, pos, slots, torch.empty(B * 300, Hq, D, dtype=dtype, device=dev()))

    token, q, q2 = make(B), torch.zeros(B, Hq, D, dtype=dtype, device=dev()), torch.zeros(B, Hq, D, dtype=dtype, device=dev())
    out, lse = torch.zeros_like(q), torch.zeros(B, Hq, device=dev())

    def step():
        slots, pos = c.reserve(1, trim=True, pos_offset=offset)
        write(c, token, pos, slots, q)
        c.attend_shared(q, tables, lens, starts, ref.scale_of(D), out, lse)

    def step_whole():
        slots, pos = whole.reserve(1)
        write(whole, token, pos, slots, q2)

    torch.cuda.synchronize()
    if graph:
        cg = torch.cuda.CUDAGraph()
        with torch.cuda.graph(cg):
            step()
    for i in range(steps):
        token.copy_(make(B))
        cg.replay() if graph else step()
        step_whole()
        torch.cuda.synchronize()
        assert torch.equal(q, q2)  # the queries are turned by the same positions
        assert not bool(c.status.any()) and not bool(whole.status.any()) and int(c.write_status) == 0
        own_len, own_table = [n + i + 1 for n in first], c.page_table.cpu()
        k, v, t, n = ref.joined(c.k_pool, c.v_pool, own_table, own_len, table, plens, start)
        assert n.tolist() == whole.seq_len.tolist()
        for r in range(B):
            m = int(n[r])
            assert torch.equal(k[r, :m], pagedref.slots(whole.k_pool, whole.page_table[r], m)), r
            assert torch.equal(v[r, :m], pagedref.slots(whole.v_pool, whole.page_table[r], m)), r
        pagedref.check_attention(out, lse, q2, whole.k_pool, whole.v_pool, whole.page_table.cpu(), whole.seq_len.cpu(),
                                 ref.scale_of(D))
