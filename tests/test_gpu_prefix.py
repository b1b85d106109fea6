"""GPU parity of shared-prefix attention with float64 attention over each request's prefix and own slots."""
import math

import pytest
import torch

import layerref as ref
import pagedref
from gpuhelp import dev

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


class Prefix:
    def __init__(self, plens, sizes, lens, Hq, Hkv, D=128, page=16, layout="slot", dtype=BF, seed=0, poison=None,
                 q_scale=2.0, start=None):
        """plens: the groups' prefixes; sizes: their requests (the rest of lens' requests belong to none)."""
        from draft_tree_build_gb300 import bastion
        self.b = bastion
        g = torch.Generator().manual_seed(seed)
        B, groups = len(lens), len(plens)
        self.plens, self.lens = list(plens), list(lens)
        self.start = start or [sum(sizes[:i]) for i in range(groups + 1)]
        need = [-(-n // page) for n in self.lens + self.plens]
        n_pages = sum(need) + 3
        ids = torch.randperm(n_pages, generator=g).tolist()

        def table(need):
            t = torch.full((len(need), max(1, max(need) + 1)), 2 ** 31 - 1, dtype=torch.int32)
            t[:, 1::2] = -1
            for r, k in enumerate(need):
                t[r, :k] = torch.tensor([ids.pop() for _ in range(k)], dtype=torch.int32)
            return t

        self.table_h, self.prefix_h = table(need[:B]), table(need[B:])
        self.k = pagedref.make_pool(n_pages, page, Hkv, D, dtype, layout, g, dev())
        self.v = pagedref.make_pool(n_pages, page, Hkv, D, dtype, layout, g, dev())
        if poison is not None:  # every slot that nobody uses
            used = torch.zeros(n_pages, page, dtype=torch.bool)
            for t, n in list(zip(self.table_h, self.lens)) + list(zip(self.prefix_h, self.plens)):
                for j in range(0, n, page):
                    used[int(t[j // page]), :min(page, n - j)] = True
            for x in (self.k, self.v):
                x.masked_fill_(~used[..., None, None].to(dev()), poison)
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev())  # noqa: E731
        self.table, self.prefix_table = self.table_h.to(dev()), self.prefix_h.to(dev())
        self.seq_len, self.prefix_len, self.group_start = i32(self.lens), i32(self.plens), i32(self.start)
        self.q = (q_scale * torch.randn(B, Hq, D, generator=g)).to(dtype).to(dev())
        self.scale = ref.scale_of(D)
        self.out, self.lse = torch.full_like(self.q, 7.0), torch.full((B, Hq), 7.0, device=dev())
        self.status = i32([0] * B)
        self.ws = bastion.workspace(bastion.bastion_paged_prefix_attention_workspace_bytes(B, Hq, Hkv, D, groups), dev())

    def run(self, ws=None, stream=None):
        self.b.bastion_paged_prefix_attention(self.q, self.k, self.v, self.table, self.seq_len, self.prefix_table,
                                              self.prefix_len, self.group_start, self.scale, self.out,
                                              self.ws if ws is None else ws, self.status, lse=self.lse, stream=stream)
        return self

    def check(self, q=None):
        torch.cuda.synchronize()
        assert int(self.status.abs().sum()) == 0
        k, v, table, lens = ref.joined(self.k, self.v, self.table_h, self.lens, self.prefix_h, self.plens, self.start)
        pagedref.check_attention(self.out, self.lse, self.q if q is None else q, k, v, table, lens, self.scale)


EDGES = [0, 1, 2, 7, 8, 9, 63, 64, 65, 127, 128, 129, 255, 256, 257, 500]


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page,layout", [(8, "slot"), (16, "head"), (32, "slot"), (64, "head"), (128, "slot")])
def test_lengths_at_every_edge(cuda_lib, dtype, D, page, layout):
    """Every prefix length with one, two and three requests of every own length."""
    sizes = [1 + i % 3 for i in range(len(EDGES))]
    lens = [EDGES[(5 * r + 3) % len(EDGES)] for r in range(sum(sizes) + 1)]
    Prefix(EDGES, sizes, lens, 8, 2, D, page, layout, dtype, seed=page + D, poison=math.nan).run().check()


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (2, 2), (6, 3), (12, 4), (10, 2), (7, 1), (32, 8), (9, 1), (24, 2), (30, 2),
                                    (16, 1), (80, 5)])
@pytest.mark.parametrize("D", [64, 128])
def test_head_groups(cuda_lib, Hq, Hkv, D):
    Prefix([300, 77], [5, 3], [10, 0, 1, 129, 40, 3, 0, 200, 17], Hq, Hkv, D, seed=Hq, poison=math.inf).run().check()


@pytest.mark.parametrize("B", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 96, 127, 128, 130, 200])
def test_rows_at_every_edge(cuda_lib, B):
    """4 to 800 query rows a KV head behind one prefix."""
    g = torch.Generator().manual_seed(B)
    lens = torch.randint(0, 60, (B,), generator=g).tolist()
    Prefix([700], [B], lens, 8, 2, 128 if B % 2 else 64, 32, seed=B, poison=math.nan).run().check()


@pytest.mark.parametrize("P,B,Hq,Hkv,D,page", [(20011, 3, 32, 8, 128, 16), (40003, 1, 8, 1, 128, 64), (9001, 70, 8, 1, 64, 8),
                                             (12345, 40, 16, 1, 128, 128), (5000, 260, 4, 2, 128, 32)])
def test_long_prefixes_are_split_and_joined(cuda_lib, P, B, Hq, Hkv, D, page):
    Prefix([P], [B], [(37 * r) % 90 for r in range(B)], Hq, Hkv, D, page, "head", HF if D == 64 else BF, seed=P).run().check()


def test_many_groups(cuda_lib):
    g = torch.Generator().manual_seed(9)
    n = 150
    sizes = torch.randint(0, 5, (n,), generator=g).tolist()
    plens = torch.randint(0, 400, (n,), generator=g).tolist()
    lens = torch.randint(0, 200, (sum(sizes) + 7,), generator=g).tolist()
    Prefix(plens, sizes, lens, 4, 2, 64, 16, seed=4, poison=math.nan).run().check()


def test_at_the_limits_of_requests_and_groups(cuda_lib):
    Prefix([20] * 1024, [1] * 1024, [r % 3 for r in range(1024)], 2, 2, 64, 8).run().check()
    Prefix([300], [1024], [r % 30 for r in range(1024)], 6, 2, 64, 8, dtype=HF).run().check()


def test_one_long_group_among_short(cuda_lib):
    Prefix([3, 30000, 200, 1], [2, 9, 1, 30], [5] * 42, 8, 2, 128, 32, "head", seed=3).run().check()


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("B", [3, 40, 100])
def test_late_maximum(cuda_lib, dtype, B):
    """Scores that rise by far more than the first tiles say, within a part and from part to part."""
    p = Prefix([3000], [B], [50] * B, 8, 2, 128, 16, dtype=dtype, seed=6, q_scale=1.0)
    for j, f in ((200, 5.0), (900, 12.0), (1500, 20.0), (2999, 28.0)):
        page, slot = int(p.prefix_h[0, j // 16]), j % 16
        p.k[page, slot] = (f * p.q[B // 2].view(2, 4, -1)[:, 1].float() / 11.3).to(dtype)
    p.run().check()


def test_flat_and_peaked_rows(cuda_lib):
    for q_scale in (0.0, 1e-3, 30.0):
        Prefix([1000, 500], [30, 40], [100] * 70, 8, 2, q_scale=q_scale, seed=12).run().check()


def test_rows_without_any_finite_score(cuda_lib):
    """A query whose scores are all -inf in the prefix, in the own slots, or in both."""
    p = Prefix([200], [3], [40, 40, 0], 4, 1, 64, 8, seed=2)
    p.q[:, :, 1:] = 0
    p.q[:, :, 0] = 1.0
    pre, mine = p.prefix_h[0, :25].long().to(dev()), p.table_h[0, :5].long().to(dev())
    p.k[pre, :, :, 0] = -math.inf
    p.k[mine, :, :, 0] = -math.inf
    p.run()
    torch.cuda.synchronize()
    # 0 times infinity is NaN: the other elements of q are 0, those of k finite, so that scores are -inf
    assert bool((p.out[0] == 0).all()) and bool(torch.isneginf(p.lse[0]).all())
    assert bool((p.out[2] == 0).all()) and bool(torch.isneginf(p.lse[2]).all())
    k, v, t, n = ref.joined(p.k, p.v, p.table_h, [40, 40, 0], p.prefix_h, [0], p.start)
    pagedref.check_attention(p.out[1:2], p.lse[1:2], p.q[1:2], k, v, t[1:2], n[1:2], p.scale)


def test_nan_stays_where_it_is_seen(cuda_lib):
    p = Prefix([300, 300], [3, 3], [20] * 6, 8, 2, 128, seed=8)
    p.q[1, 2] = math.nan
    p.run()
    torch.cuda.synchronize()
    seen = p.out.isnan().all(-1)
    assert bool(seen[1, 2]) and int(seen.sum()) == 1 and int(p.out.isnan().any(-1).sum()) == 1
    q = p.q.clone()
    q[1, 2] = 0
    p.out[1, 2], p.lse[1, 2], p.q = 0, 0, q
    keep = [0, 2, 3, 4, 5]
    k, v, t, n = ref.joined(p.k, p.v, p.table_h, p.lens, p.prefix_h, p.plens, p.start)
    pagedref.check_attention(p.out[keep].contiguous(), p.lse[keep], q[keep], k, v, t[keep], n[keep], p.scale)


def test_strided_queries_shared_pool_and_in_place(cuda_lib):
    p = Prefix([500], [20], [33] * 20, 8, 2, 128, seed=1)
    wide = torch.zeros(20, 3, 8, 128, dtype=BF, device=dev())
    wide[:, 1] = p.q
    q = p.q.clone()
    both = torch.stack([p.k, p.v], 2)  # keys and values of a slot side by side
    p.k, p.v, p.q = both[:, :, 0], both[:, :, 1], wide[:, 1]
    p.run().check()
    p.q = q.clone()
    p.out = p.q
    p.run().check(q)


def test_offsets_past_32_bits(cuda_lib):
    """Pages more than 2^31 elements into the pool."""
    page, H, D, n = 128, 2, 128, 70000
    k = torch.zeros(n, page, H, D, dtype=BF, device=dev())
    v = torch.zeros_like(k)
    p = Prefix([300], [4], [40] * 4, 8, 2, 128, page, seed=5)
    far = n - 1 - torch.arange(p.k.shape[0], device=dev())
    k[far], v[far] = p.k, p.v
    p.k, p.v = k, v
    p.table_h, p.prefix_h = (torch.where((t >= 0) & (t < 1000), n - 1 - t, t) for t in (p.table_h, p.prefix_h))
    p.table, p.prefix_table = p.table_h.to(dev()), p.prefix_h.to(dev())
    p.run().check()


def test_repeats_bit_for_bit_and_shares_a_workspace(cuda_lib):
    big, small = Prefix([9000, 700], [40, 9], [100] * 49, 8, 2), Prefix([50], [3], [0, 1, 2], 4, 4, 64, dtype=HF)
    ws = max(big.ws, small.ws, key=lambda x: x.numel())
    big.run(ws)
    torch.cuda.synchronize()
    out, lse = big.out.clone(), big.lse.clone()
    for _ in range(10):
        small.run(ws)
        big.run(ws)
        torch.cuda.synchronize()
        assert torch.equal(big.out, out) and torch.equal(big.lse, lse)
    small.check()
    big.check()


def test_on_streams_and_in_graphs(cuda_lib):
    a, b = Prefix([2000], [30], [100] * 30, 8, 2), Prefix([100, 900], [4, 5], [9] * 9, 8, 1, 64)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(10):
        a.run(stream=s1)
        b.run(stream=s2)
    a.check()
    b.check()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a.run()
        b.run()
    a.q.normal_()
    a.lens, a.plens, a.start = [3 * r for r in range(30)], [1234], [2, 27]
    for t, x in ((a.seq_len, a.lens), (a.prefix_len, a.plens), (a.group_start, a.start)):
        t.copy_(torch.tensor(x, dtype=torch.int32))
    for _ in range(3):
        g.replay()
    a.check()
    b.check()


def test_status(cuda_lib):
    def fresh():
        return Prefix([100, 50, 60], [2, 2, 2], [10] * 6, 4, 2, 64)

    def status(p):
        p.run()
        torch.cuda.synchronize()
        return p.status.tolist()

    p = fresh()
    p.prefix_len[1] = 10 ** 6
    assert status(p)[2] & 8
    p = fresh()
    p.prefix_len[1] = -1
    assert status(p) == [0, 0, 8, 0, 0, 0]
    p = fresh()
    p.prefix_table[2, 3] = 10 ** 6  # in use: slots 48..59
    assert status(p) == [0, 0, 0, 0, 64, 0]
    p = fresh()
    p.table[3, 0] = -1
    assert status(p) == [0, 0, 0, 64, 0, 0]
    p = fresh()
    p.seq_len[5] = 10 ** 6
    assert status(p)[5] & 8
    for start, told in (([0, 2, 1, 6], 2), ([0, 2, 4, 7], 4), ([-1, 2, 4, 6], 0), ([0, -3, 4, 6], 0),
                        ([9, 2, 4, 6], 5)):
        p = fresh()
        p.group_start.copy_(torch.tensor(start, dtype=torch.int32))
        got = status(p)
        assert got[told] == 512, (start, got)
    # a group that is left out: its requests attend to their own slots, the others as ever
    p = Prefix([100, 50, 60], [2, 2, 2], [10] * 6, 4, 2, 64, start=[0, 2, 4, 7])
    p.run()
    torch.cuda.synchronize()
    p.status.zero_()
    p.check()


def test_groups_that_overlap(cuda_lib):
    """A request of two groups belongs to the first; nothing is written out of place."""
    p = Prefix([100, 50, 600], [2, 2, 2], [10] * 6, 4, 2, 64, start=[0, 5, 3, 6])
    p.run()
    torch.cuda.synchronize()
    assert int(p.status.sum()) == 512
    p.status.zero_()
    p.check()


def test_agrees_with_plain_paged_attention(cuda_lib):
    """The same requests through bastion_paged_attention, with the prefix's pages in every request's table."""
    p = Prefix([512], [12], [60] * 12, 32, 8, 128, 16, seed=21)
    p.run().check()
    table = torch.cat([p.prefix_table[:, :32].expand(12, 32), p.table[:, :4]], 1).contiguous()
    out, lse = torch.zeros_like(p.out), torch.zeros_like(p.lse)
    ws = p.b.workspace(p.b.bastion_paged_attention_workspace_bytes(12, 32, 8, 128, 36 * 16, False), dev())
    p.b.bastion_paged_attention(p.q, p.k, p.v, table, p.seq_len + 512, p.scale, out, ws, p.status, lse=lse)
    torch.cuda.synchronize()
    assert float((p.lse - lse).abs().max()) < 1e-5
    assert float((p.out.float() - out.float()).abs().max()) <= 2 ** -7 * float(out.float().abs().max())


@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 128), (8, 1, 64), (12, 1, 128), (3, 1, 64)])
@pytest.mark.parametrize("own", [40, 48, 49, 64, 65, 300, 512, 1008, 1009, 1025, 3000])
def test_short_and_long_own_slots(cuda_lib, Hq, Hkv, D, own):
    """On both sides of the sizes up to which own slots have a kernel of their own."""
    lens = [own, 0, 1, own // 2, min(own, 129), own - 1, min(own, 17)]
    for dtype in (BF, HF):
        Prefix([300, 1500], [3, 3], lens, Hq, Hkv, D, 16, "head", dtype, seed=own + Hq, poison=math.nan).run().check()


def test_long_own_slots_in_graphs_and_in_place(cuda_lib):
    a = Prefix([2000], [30], [50 * r for r in range(30)], 8, 2, seed=31)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a.run()
    a.q.normal_()
    for _ in range(3):
        g.replay()
    a.check()
    q = a.q.clone()
    a.out = a.q
    a.run().check(q)
