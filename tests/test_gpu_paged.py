"""GPU parity of the paged cache (append, one-token attention with accumulated
weights, eviction) with plain references: attention in float64, copies and
selections exactly."""
import math

import pytest
import torch

import pagedref as ref
from gpuhelp import dev

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _table(lens, page, gen, spare=3, garbage=True):
    """Pages anywhere in the pool; entries past a request's last used page hold no page numbers."""
    lens = [int(n) for n in lens]
    max_pages = max(1, max(-(-n // page) for n in lens) + 1)
    need = [-(-n // page) for n in lens]
    n_pages = sum(need) + spare
    ids = torch.randperm(n_pages, generator=gen)
    t = torch.full((len(lens), max_pages), -1, dtype=torch.int32)
    if garbage:
        t[:, ::2] = 2 ** 31 - 1
    at = 0
    for r, k in enumerate(need):
        t[r, :k] = ids[at:at + k].to(torch.int32)
        at += k
    return t, n_pages


def _poison(pool, table, lens, value):
    """Every slot that no request uses gets the value."""
    page = pool.shape[1]
    used = torch.zeros(pool.shape[:2], dtype=torch.bool)
    for r, n in enumerate(lens):
        for j in range(int(n)):
            used[int(table[r, j // page]), j % page] = True
    pool.masked_fill_(~used[..., None, None].to(pool.device), value)


class Case:
    """One attention call's tensors."""

    def __init__(self, lens, Hq, Hkv, D=128, page=16, layout="slot", dtype=BF, weights=False, seed=0, q_scale=2.0,
                 poison=None):
        from draft_tree_build_gb300 import bastion
        self.b = bastion
        g = _gen(seed)
        self.lens = torch.tensor(lens, dtype=torch.int32)
        t, n_pages = _table(lens, page, g)
        self.k = ref.make_pool(n_pages, page, Hkv, D, dtype, layout, g, dev())
        self.v = ref.make_pool(n_pages, page, Hkv, D, dtype, layout, g, dev())
        if poison is not None:
            _poison(self.k, t, lens, poison)
            _poison(self.v, t, lens, poison)
        self.table, self.seq_len = t.to(dev()), self.lens.to(dev())
        B = len(lens)
        self.q = (q_scale * torch.randn(B, Hq, D, generator=g)).to(dtype).to(dev())
        self.scale = 1 / math.sqrt(D)
        self.out = torch.full_like(self.q, 7.0)
        self.lse = torch.full((B, Hq), 7.0, device=dev())
        cap = t.shape[1] * page
        self.acc = torch.rand(B, Hkv, cap, generator=g).to(dev()) if weights else None
        self.acc_out = torch.full((B, Hkv, cap), 7.0, device=dev()) if weights else None
        self.status = torch.zeros(B, dtype=torch.int32, device=dev())
        self.ws = bastion.workspace(bastion.bastion_paged_attention_workspace_bytes(B, Hq, Hkv, D, cap, weights),
                                    dev())

    def run(self, ws=None, stream=None, acc_out=None):
        self.b.bastion_paged_attention(self.q, self.k, self.v, self.table, self.seq_len, self.scale, self.out,
                                       self.ws if ws is None else ws, self.status, lse=self.lse, acc=self.acc,
                                       acc_out=self.acc_out if acc_out is None else acc_out, stream=stream)
        return self

    def check(self):
        torch.cuda.synchronize()
        assert int(self.status.abs().sum()) == 0
        ref.check_attention(self.out, self.lse, self.q, self.k, self.v, self.table, self.lens, self.scale,
                            self.acc, self.acc_out, 7.0)


EDGES = [0, 1, 2, 7, 8, 9, 63, 64, 65, 127, 128, 129, 255, 256, 257, 500, 0, 1000]


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page,layout", [(8, "slot"), (16, "head"), (32, "slot"), (64, "slot"), (128, "head")])
def test_attention_lengths_at_every_edge(cuda_lib, dtype, D, page, layout):
    Case(EDGES, 8, 2, D, page, layout, dtype, weights=True, seed=page + D, poison=float("nan")).run().check()


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (2, 2), (6, 3), (12, 4), (10, 2), (12, 2), (7, 1), (32, 4), (9, 1),
                                    (24, 2), (30, 2), (16, 1), (80, 5)])
@pytest.mark.parametrize("D", [64, 128])
def test_attention_head_groups(cuda_lib, Hq, Hkv, D):
    Case([300, 1, 129, 0], Hq, Hkv, D, weights=True, seed=Hq, poison=float("inf")).run().check()


@pytest.mark.parametrize("B,n,Hq,Hkv,page", [(1, 70001, 32, 8, 64), (1, 40003, 8, 1, 16), (2, 20011, 16, 1, 8),
                                             (3, 9001, 32, 8, 16)])
def test_attention_long_rows_are_split_and_joined(cuda_lib, B, n, Hq, Hkv, page):
    lens = [max(1, n - 1234 * i) for i in range(B)]
    Case(lens, Hq, Hkv, 128, page, weights=True, seed=n).run().check()


def test_attention_many_requests(cuda_lib):
    g = _gen(5)
    lens = torch.randint(0, 400, (700,), generator=g).tolist()
    Case(lens, 8, 2, 64, 16, weights=True, seed=3).run().check()


@pytest.mark.parametrize("B,Hq,Hkv", [(1024, 3, 3), (255, 257, 257)])
def test_attention_at_the_limits_of_requests_and_heads(cuda_lib, B, Hq, Hkv):
    """1,024 requests; 65,535 (request, KV head) pairs, one unit each."""
    lens = torch.randint(0, 12 if Hkv > 3 else 150, (B,), generator=_gen(B)).tolist()
    Case(lens, Hq, Hkv, 64, 8, weights=True, seed=B).run().check()


def test_attention_one_long_among_many_short(cuda_lib):
    lens = [3] * 40 + [30000] + [0, 5] * 20
    Case(lens, 16, 4, 128, 32, weights=True, seed=4).run().check()


@pytest.mark.parametrize("dtype", [BF, HF])
def test_attention_late_maximum(cuda_lib, dtype):
    """Scores that exceed every earlier one far into the row, twice, and by little steps."""
    c = Case([3000, 700], 8, 2, 128, 16, dtype=dtype, weights=True, seed=6)
    u = torch.randn(128, generator=_gen(9)).to(dev())
    u /= u.norm()
    c.q += (3.0 * u).to(dtype)
    page = 16
    for r, j, f in [(0, 1500, 12.0), (0, 2900, 40.0), (1, 650, 25.0)] + [(0, 200 * i, 2.0 * i) for i in range(1, 7)]:
        c.k[int(c.table[r, j // page]), j % page] = (f * u).to(dtype)
    c.run().check()


def test_attention_flat_and_peaked_rows(cuda_lib):
    """Zero queries give the mean of v; a large scale gives one slot's v."""
    c = Case([777, 130], 4, 2, seed=7, weights=True)
    c.q.zero_()
    c.run().check()
    c = Case([777, 130], 4, 2, seed=8, weights=True, q_scale=30.0)
    c.run().check()


def test_attention_minus_infinity_scores(cuda_lib):
    """Keys of -inf against queries that are positive there: those slots weigh nothing; a head that sees
    only such slots is empty."""
    c = Case([300, 40], 4, 2, seed=10, weights=True)
    c.q.abs_()
    keep = c.k.clone()
    for j in range(40):  # request 1: all of its slots
        c.k[int(c.table[1, j // 16]), j % 16, :, 5] = -math.inf
    for j in range(0, 300, 3):
        c.k[int(c.table[0, j // 16]), j % 16, :, 5] = -math.inf
    c.run()
    torch.cuda.synchronize()
    assert bool((c.out[1] == 0).all()) and bool(torch.isneginf(c.lse[1]).all())
    assert torch.equal(c.acc_out[1, :, :40], c.acc[1, :, :40])
    live = [j for j in range(300) if j % 3]
    k = ref.slots(keep, c.table[0], 300)[live].double()
    v = ref.slots(c.v, c.table[0], 300)[live].double()
    s = torch.einsum("hgd,lhd->hgl", c.q[0].double().view(2, 2, 128), k) * c.scale
    out = torch.einsum("hgl,lhd->hgd", s.softmax(-1), v).view(4, 128)
    size = torch.einsum("hgl,lhd->hgd", s.softmax(-1), v.abs()).view(4, 128)
    mag = torch.einsum("hgd,lhd->hgl", c.q[0].double().abs().view(2, 2, 128), k.abs()).amax() * c.scale
    err = (c.out[0].double() - out).abs()
    assert bool((err <= 2.0 ** -8 * out.abs() * 1.01 + size * (2.0 ** -15 * mag + 2.0 ** -14)).all())
    assert torch.equal(c.acc_out[0, :, 0:300:3], c.acc[0, :, 0:300:3])


def test_attention_nan_stays_in_its_head(cuda_lib):
    c = Case([300, 40], 8, 2, seed=11)
    clean = c.run().out.clone()
    c.k[int(c.table[0, 100 // 16]), 100 % 16, 1, 3] = float("nan")  # KV head 1 of request 0
    c.q[1, 2, 0] = float("nan")                                      # one query head of request 1
    c.run()
    torch.cuda.synchronize()
    bad = torch.zeros(2, 8, dtype=torch.bool, device=dev())
    bad[0, 4:] = True
    bad[1, 2] = True
    assert bool(torch.isnan(c.out[bad]).all())
    assert torch.equal(c.out[~bad], clean[~bad])


def test_attention_strided_queries_and_shared_pool(cuda_lib):
    """q as a slice of a fused projection; K and V interleaved in one allocation."""
    c = Case([300, 17, 129], 8, 2, 128, 16, weights=True, seed=12)
    both = torch.stack([c.k, c.v], 1).contiguous()  # [pages, 2, page, Hkv, D]
    c.k, c.v = both[:, 0], both[:, 1]
    fused = torch.randn(3, 8 + 4, 128, device=dev()).to(BF)
    fused[:, :8] = c.q
    c.q = fused[:, :8]
    assert c.q.stride(0) != 8 * 128
    c.run().check()


def test_attention_pools_in_any_order_of_dimensions(cuda_lib):
    """Pages nearer to one another than a page's slots; heads outermost."""
    for order in ((1, 0, 2, 3), (2, 0, 1, 3), (2, 1, 0, 3)):
        c = Case([300, 17, 129], 8, 2, 128, 16, weights=True, seed=30, poison=float("nan"))
        back = [order.index(i) for i in range(4)]
        c.k, c.v = (x.permute(order).contiguous().permute(back) for x in (c.k, c.v))
        assert not c.k.is_contiguous()
        c.run().check()


def test_attention_repeated_pages(cuda_lib):
    """Requests that share pages, and one that lists a page twice."""
    c = Case([300, 300, 64], 8, 2, 128, 16, weights=True, seed=31)
    c.table[1] = c.table[0]
    c.table[2, 1:4] = c.table[2, 0]
    c.run().check()


def test_attention_offsets_past_32_bits(cuda_lib):
    """Pools of more than 2^31 elements; the requests' pages lie at both ends."""
    from draft_tree_build_gb300 import bastion
    n_pages, page, Hkv, D = 16500, 128, 8, 128
    assert n_pages * page * Hkv * D > 2 ** 31
    k = torch.empty(n_pages, page, Hkv, D, dtype=BF, device=dev())
    v = torch.empty_like(k)
    ids = [n_pages - 1, 0, n_pages - 2, 1]
    for i in ids:
        k[i].normal_()
        v[i].normal_()
    table = torch.tensor([ids[:2], ids[2:]], dtype=torch.int32, device=dev())
    lens = torch.tensor([200, 255], dtype=torch.int32)
    q = torch.randn(2, 16, D, device=dev()).to(BF)
    out, lse = torch.empty_like(q), torch.empty(2, 16, device=dev())
    st = torch.zeros(2, dtype=torch.int32, device=dev())
    ws = bastion.workspace(bastion.bastion_paged_attention_workspace_bytes(2, 16, Hkv, D, 256, False), dev())
    bastion.bastion_paged_attention(q, k, v, table, lens.to(dev()), 0.1, out, ws, st, lse=lse)
    torch.cuda.synchronize()
    ref.check_attention(out, lse, q, k, v, table, lens, 0.1)


def test_attention_repeats_bit_for_bit_and_shares_a_workspace(cuda_lib):
    """The same call gives the same bits; calls of other sizes may use the workspace in between."""
    from draft_tree_build_gb300 import bastion
    big = Case([20000, 3, 5000], 32, 8, weights=True, seed=13)
    small = Case([40, 700], 16, 1, 64, weights=True, seed=14)
    n = max(big.ws.numel(), small.ws.numel())
    ws = bastion.workspace(n, dev())
    big.run(ws)
    first = [t.clone() for t in (big.out, big.lse, big.acc_out)]
    for _ in range(5):
        small.run(ws)
        big.run(ws)
        small.check()
    big.check()
    for a, b in zip(first, (big.out, big.lse, big.acc_out)):
        assert torch.equal(a, b)


def test_both_ways_into_the_library_agree(cuda_lib, monkeypatch):
    """With and without the compiled short way: the same results, and refusals from the same checks."""
    from draft_tree_build_gb300 import bastion

    def all_calls():
        a = Case([700, 0, 90], 8, 2, 128, 16, layout="head", weights=True, seed=50).run(stream=torch.cuda.Stream())
        c = Cache([90, 64, 30], 20, Hkv=2, D=64, page=8, seed=51)
        _positions(c)
        c.evict(60, 2, 8, False)
        c.append(*c.rows(5), rows=torch.tensor([[0, 2, -1], [4, -1, -1], [1, 1, 1]], dtype=torch.int32))
        c.same()
        a.check()
        return [a.out, a.lse, a.acc_out, c.g_k, c.g_v, c.g_acc, c.g_pos, c.g_lens, c.g_seen]

    assert bastion._marshal is not None
    calls = []
    with monkeypatch.context() as mp:
        spy = type("Spy", (), {n: (lambda *x, f=getattr(bastion._marshal, n): calls.append(f(*x)) or calls[-1])
                               for n in ("append", "attention", "evict")})
        mp.setattr(bastion, "_marshal", spy)
        first = all_calls()
    assert calls == [0, 0, 0]  # all three were taken
    monkeypatch.setattr(bastion, "_marshal", None)
    for x, y in zip(first, all_calls()):
        assert torch.equal(x, y)
    c = Case([40], 4, 2, seed=52)
    for marshal in (None, bastion._load_marshal(bastion.lib())):
        monkeypatch.setattr(bastion, "_marshal", marshal)
        lens = c.seq_len
        c.seq_len = lens.long()
        with pytest.raises(bastion.BastionError, match="seq_len"):
            c.run()
        c.seq_len, scale = lens, c.scale
        c.scale = -1.0
        with pytest.raises(bastion.BastionError, match="out of range"):
            c.run()
        c.scale = scale
        c.run().check()


def test_one_workspace_serves_all_calls(cuda_lib):
    """Attention, eviction and append in turn on one workspace, whatever they leave in it."""
    from draft_tree_build_gb300 import bastion
    a = Case([20000, 3, 5000], 32, 8, weights=True, seed=40)
    c = Cache([900, 700, 300, 40], 130, Hkv=8, D=64, page=8, seed=41)
    _positions(c)
    ws = bastion.workspace(max(a.ws.numel(), c.ws.numel()), dev())
    c.ws = ws
    for budget in (600, 350, 60):
        a.run(ws)
        c.evict(budget, 2, 20)
        c.append(*c.rows(5))
        a.run(ws)
        a.check()
        c.same()
    assert int(c.status.sum()) == 0


def test_attention_output_in_place_of_the_queries(cuda_lib):
    c = Case([300, 0, 5000, 1], Hq=8, Hkv=2, seed=21).run()
    q = c.q.clone()
    c.b.bastion_paged_attention(q, c.k, c.v, c.table, c.seq_len, c.scale, q, c.ws, c.status)
    c.check()
    assert torch.equal(q, c.out)


def test_attention_weights_in_place(cuda_lib):
    c = Case([300, 0, 77], 8, 4, weights=True, seed=15).run()
    acc = c.acc.clone()
    c.run(acc_out=acc)  # not in place: c.acc is the input
    torch.cuda.synchronize()
    inplace = c.acc.clone()
    c.b.bastion_paged_attention(c.q, c.k, c.v, c.table, c.seq_len, c.scale, c.out, c.ws, c.status, lse=c.lse,
                                acc=inplace, acc_out=inplace)
    torch.cuda.synchronize()
    assert torch.equal(inplace, acc)


def test_attention_on_streams_and_in_graphs(cuda_lib):
    """Two calls at once on two streams with a workspace each; a captured call replayed on new inputs."""
    a, b = Case([5000, 20], 8, 2, weights=True, seed=16), Case([900] * 9, 8, 1, 64, weights=True, seed=17)
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
    a.lens = torch.tensor([123, 4000], dtype=torch.int32)
    a.lens[1] = min(4000, a.table.shape[1] * 16)
    a.table[1] = a.table[0]  # shared, read-only pages
    a.seq_len.copy_(a.lens)
    a.acc_out.fill_(7.0)
    for _ in range(3):
        g.replay()
    a.check()
    b.check()


def test_attention_status(cuda_lib):
    from draft_tree_build_gb300 import bastion
    c = Case([300, 40, 500], 8, 2, seed=18)
    clean = c.run().out.clone()
    c.table[1, 1] = -3
    c.seq_len[2] = c.table.shape[1] * 16 + 1
    c.run()
    torch.cuda.synchronize()
    st = c.status.tolist()
    assert st[0] == 0 and st[1] == bastion.STATUS_BAD_PAGE and st[2] & bastion.STATUS_KV_OVERFLOW
    assert torch.equal(c.out[0], clean[0])
    c.status.zero_()
    c.seq_len[2] = -1
    c.run()
    torch.cuda.synchronize()
    assert c.status.tolist()[2] == bastion.STATUS_KV_OVERFLOW


# --------------------------------------------------------------------------- append

class Cache:
    """A cache with its bookkeeping on the GPU and a copy on the CPU."""

    def __init__(self, lens, max_pages, Hkv=2, D=64, page=8, layout="slot", dtype=BF, seed=0, seen=None):
        from draft_tree_build_gb300 import bastion
        self.b = bastion
        g = _gen(seed)
        B = len(lens)
        self.B, self.Hkv, self.D, self.page, self.cap = B, Hkv, D, page, max_pages * page
        n_pages = B * max_pages + 2
        self.table = torch.randperm(n_pages, generator=g)[: B * max_pages].view(B, max_pages).to(torch.int32)
        self.k = ref.make_pool(n_pages, page, Hkv, D, dtype, layout, g, "cpu")
        self.v = ref.make_pool(n_pages, page, Hkv, D, dtype, layout, g, "cpu")
        self.lens = torch.tensor(lens, dtype=torch.int32)
        self.seen = torch.tensor(lens if seen is None else seen, dtype=torch.int32)
        self.acc = torch.rand(B, Hkv, self.cap, generator=g)
        self.pos = torch.randint(0, 1000, (B, Hkv, self.cap), generator=g, dtype=torch.int32)
        self.gen = g
        self.to_gpu()

    def to_gpu(self):
        for n in ("k", "v", "table", "lens", "seen", "acc", "pos"):
            setattr(self, "g_" + n, getattr(self, n).to(dev()))  # .to keeps a permuted view's strides
        self.status = torch.zeros(self.B, dtype=torch.int32, device=dev())
        self.ws = self.b.workspace(max(self.b.bastion_paged_append_workspace_bytes(self.B),
                                       self.b.bastion_paged_evict_workspace_bytes(self.B, self.Hkv, self.cap)), dev())

    def same(self, names=("k", "v", "lens", "seen", "acc", "pos")):
        torch.cuda.synchronize()
        for n in names:
            a, b = getattr(self, n), getattr(self, "g_" + n).cpu()
            if n == "acc":
                a, b = a.view(torch.int32), b.view(torch.int32)
            assert torch.equal(a, b), n

    def append(self, k_new, v_new, rows=None, n_new=None):
        to = lambda t: None if t is None else t.to(dev())  # noqa: E731
        self.b.bastion_paged_append(k_new.to(dev()), v_new.to(dev()), self.g_k, self.g_v, self.g_table, self.g_lens,
                                    self.g_lens, self.ws, self.status, rows=to(rows), n_new=to(n_new),
                                    acc=self.g_acc, pos=self.g_pos, n_seen=self.g_seen, n_seen_out=self.g_seen)
        self.lens, self.seen = ref.append(k_new, v_new, self.k, self.v, self.table, self.lens, self.seen, self.acc,
                                          self.pos, rows, n_new)

    def rows(self, n, dtype=BF):
        f = lambda: torch.randn(self.B, n, self.Hkv, self.D, generator=self.gen).to(dtype)  # noqa: E731
        return f(), f()

    def evict(self, budget, sink, recent, inplace=True):
        acc_out = self.g_acc if inplace else torch.full_like(self.g_acc, 7.0)
        pos_out = self.g_pos if inplace else torch.full_like(self.g_pos, 7)
        len_out = self.g_lens if inplace else torch.full_like(self.g_lens, 7)
        self.b.bastion_paged_evict(self.g_k, self.g_v, self.g_table, self.g_lens, self.g_seen, self.g_acc, self.g_pos,
                                   budget, sink, recent, len_out, acc_out, pos_out, self.ws, self.status)
        a, p = (self.acc, self.pos) if inplace else (torch.full_like(self.acc, 7.0), torch.full_like(self.pos, 7))
        self.lens = ref.evict(self.k, self.v, self.table, self.lens, self.seen, self.acc, self.pos, budget, sink,
                              recent, a, p)
        self.acc, self.pos, self.g_acc, self.g_pos, self.g_lens = a, p, acc_out, pos_out, len_out


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("D,page,layout,Hkv", [(64, 8, "slot", 3), (128, 16, "head", 8), (128, 128, "slot", 1)])
def test_append_one_token_and_prompts(cuda_lib, dtype, D, page, layout, Hkv):
    c = Cache([0, 1, page - 1, page, 37], 128 // page + 3, Hkv, D, page, layout, dtype, seed=page)
    c.append(*c.rows(1, dtype))
    c.same()
    c.append(*c.rows(70, dtype), n_new=torch.tensor([70, 0, -5, 1, 33], dtype=torch.int32))
    c.same()
    assert int(c.status.sum()) == 0


def test_append_accepted_paths(cuda_lib):
    c = Cache([5, 0, 30, 16], 8, seed=2, seen=[100, 0, 31, 400])
    rows = torch.tensor([[0, 3, 7, 12, -1, -1], [0, -1, 4, 4, 4, 4], [-1, 0, 1, 2, 3, 4], [0, 1, 2, 3, 4, 15]],
                        dtype=torch.int32)
    c.append(*c.rows(16), rows=rows)
    c.same()
    c.append(*c.rows(16), rows=rows, n_new=torch.tensor([2, 9, 1, 0], dtype=torch.int32))
    c.same()
    assert int(c.status.sum()) == 0


def test_append_full_cache_and_bad_rows(cuda_lib):
    from draft_tree_build_gb300 import bastion
    c = Cache([60, 64, 57, 10], 8, seed=3)
    k, v = c.rows(7)
    c.append(k, v)  # requests 0 and 1 do not fit, 2 just does
    c.same()
    assert c.status.tolist() == [bastion.STATUS_KV_OVERFLOW] * 2 + [0, 0]
    c.status.zero_()
    before = c.g_k.clone()
    rows = torch.tensor([[-1], [-1], [-1], [7]], dtype=torch.int32)  # row 7 of 7
    c.b.bastion_paged_append(k.to(dev()), v.to(dev()), c.g_k, c.g_v, c.g_table, c.g_lens, c.g_lens, c.ws, c.status,
                             rows=rows.to(dev()))
    torch.cuda.synchronize()
    assert c.status.tolist() == [0, 0, 0, bastion.STATUS_BAD_ROW]
    assert torch.equal(before, c.g_k)
    c.status.zero_()
    c.g_table[3] = c.k.shape[0]  # no such page
    c.b.bastion_paged_append(k.to(dev()), v.to(dev()), c.g_k, c.g_v, c.g_table, c.g_lens, c.g_lens, c.ws, c.status,
                             n_new=torch.tensor([0, 0, 0, 3], dtype=torch.int32, device=dev()))
    torch.cuda.synchronize()
    assert c.status.tolist() == [0, 0, 0, bastion.STATUS_BAD_PAGE]
    assert torch.equal(before, c.g_k)


def test_append_strided_rows_and_separate_lengths(cuda_lib):
    """K and V as slices of a fused projection; lengths written to other arrays; no bookkeeping."""
    c = Cache([5, 11, 0], 6, Hkv=2, D=64, seed=4)
    qkv = torch.randn(3, 9, 8, 64, generator=c.gen).to(BF)
    k, v = qkv[:, :, 4:6], qkv[:, :, 6:8]
    g = qkv.to(dev())
    out = torch.full((3,), -1, dtype=torch.int32, device=dev())
    c.b.bastion_paged_append(g[:, :, 4:6], g[:, :, 6:8], c.g_k, c.g_v, c.g_table, c.g_lens, out, c.ws, c.status)
    new, _ = ref.append(k, v, c.k, c.v, c.table, c.lens, c.seen, None, None)
    c.same()
    assert torch.equal(out.cpu(), new)


def test_append_one_token_of_any_stride(cuda_lib):
    """One token's keys as a transposed view (heads before tokens), its values not."""
    c = Cache([5, 0, 61], 12, Hkv=4, seed=8)
    k, v = c.rows(1)
    k_t = k.transpose(1, 2).clone(memory_format=torch.contiguous_format).to(dev()).transpose(1, 2)
    v_g = v.to(dev())
    assert k_t.stride() != v_g.stride()
    c.b.bastion_paged_append(k_t, v_g, c.g_k, c.g_v, c.g_table, c.g_lens, c.g_lens, c.ws, c.status)
    c.lens, _ = ref.append(k, v, c.k, c.v, c.table, c.lens, c.seen, None, None)
    c.same(("k", "v", "lens"))


def test_append_one_array_of_lengths(cuda_lib):
    """Without evictions a request's tokens are its slots: seq_len serves as n_seen."""
    c = Cache([5, 0, 61], 12, seed=7)
    k, v = c.rows(20)
    c.b.bastion_paged_append(k.to(dev()), v.to(dev()), c.g_k, c.g_v, c.g_table, c.g_lens, c.g_lens, c.ws, c.status,
                             acc=c.g_acc, pos=c.g_pos, n_seen=c.g_lens, n_seen_out=c.g_lens)
    c.lens, _ = ref.append(k, v, c.k, c.v, c.table, c.lens, c.seen, c.acc, c.pos)
    c.same(("k", "v", "lens", "acc", "pos"))


def test_append_long_prompts(cuda_lib):
    c = Cache([100, 0], 300, Hkv=4, D=128, page=16, seed=5)
    c.append(*c.rows(4501), n_new=torch.tensor([4501, 1777], dtype=torch.int32))
    c.same()


# --------------------------------------------------------------------------- eviction

def _positions(c):
    """Distinct positions per head in a shuffled order."""
    for r in range(c.B):
        for h in range(c.Hkv):
            c.pos[r, h] = torch.randperm(c.cap, generator=c.gen).to(torch.int32)
    c.seen = torch.full((c.B,), c.cap, dtype=torch.int32)
    c.to_gpu()


@pytest.mark.parametrize("inplace", [True, False])
@pytest.mark.parametrize("budget,sink,recent", [(1, 0, 0), (1, 1, 0), (40, 0, 0), (40, 4, 16), (64, 60, 4), (100, 8, 50),
                                                (500, 2, 20)])
def test_evict_keeps_the_heaviest(cuda_lib, budget, sink, recent, inplace):
    c = Cache([0, 1, 40, 41, 64, 100, 101, 300], 40, Hkv=3, D=64, page=8, seed=budget + sink)
    _positions(c)
    c.evict(budget, sink, recent, inplace)
    c.same()
    assert int(c.status.sum()) == 0


@pytest.mark.parametrize("D,page,layout,dtype", [(128, 16, "head", BF), (128, 64, "slot", HF)])
def test_evict_long(cuda_lib, D, page, layout, dtype):
    c = Cache([9000, 5000, 2049], 9216 // page, Hkv=2, D=D, page=page, layout=layout, dtype=dtype, seed=page)
    _positions(c)
    c.evict(2048, 4, 256)
    c.same()


def test_evict_more_slots_than_a_cluster_holds(cuda_lib):
    """380,000 slots: the keys of a head do not fit the shared memory of eight CTAs."""
    c = Cache([380000, 379999], 2970, Hkv=1, D=64, page=128, seed=26)
    _positions(c)
    c.evict(379000, 4, 1000)
    c.same()
    c.evict(100, 4, 10, False)
    c.same()


def test_evict_no_spread_in_the_weights(cuda_lib):
    """Long runs of equal and nearly equal weights: the deciding bin holds almost every slot."""
    c = Cache([20000, 20000, 9000], 1250, Hkv=2, D=64, page=16, seed=27)
    c.acc[0] = 0.0
    c.acc[1] = 1.0 + torch.randint(0, 3000, c.acc[1].shape, generator=c.gen) * 2.0 ** -23
    c.acc[2, :, ::2] = 0.5
    _positions(c)
    c.evict(4000, 4, 100)
    c.same()


def test_evict_ties_go_to_the_lower_slot(cuda_lib):
    c = Cache([300, 299, 64], 40, Hkv=2, D=64, seed=21)
    c.acc = (c.acc * 4).floor()  # four values
    c.acc[1] = 0.25              # all alike
    c.acc[2] = -c.acc[2]         # negative, and -0.0
    _positions(c)
    c.evict(60, 2, 9)
    c.same()


def test_evict_extreme_weights(cuda_lib):
    from draft_tree_build_gb300 import bastion
    c = Cache([300, 300], 40, Hkv=2, D=64, seed=22)
    c.acc[0, 0, ::7] = math.inf
    c.acc[0, 1, ::7] = -math.inf
    c.acc[1] = torch.finfo(torch.float32).tiny * torch.rand(2, c.cap, generator=c.gen)  # subnormals among them
    _positions(c)
    c.evict(100, 0, 10)
    c.same()
    assert int(c.status.sum()) == 0
    c = Cache([300, 300], 40, Hkv=2, D=64, seed=23)
    c.acc[0, 1, 5::50] = float("nan")
    _positions(c)
    c.evict(100, 0, 10)
    c.same()
    assert c.status.tolist() == [bastion.STATUS_NONFINITE, 0]


def test_evict_more_protected_than_budget(cuda_lib):
    """Equal positions: every slot is protected, the lower slots stay."""
    c = Cache([200], 40, Hkv=2, D=64, seed=24)
    c.pos.fill_(5)
    c.to_gpu()
    c.evict(50, 10, 0)
    c.same()


def test_evict_status(cuda_lib):
    from draft_tree_build_gb300 import bastion
    c = Cache([200, 200, 200], 40, Hkv=2, D=64, seed=25)
    _positions(c)
    c.g_table[0] = -1
    c.g_lens[2] = c.cap + 1
    before = c.g_k.clone()
    b = c.b
    b.bastion_paged_evict(c.g_k, c.g_v, c.g_table, c.g_lens, c.g_seen, c.g_acc, c.g_pos, 300, 0, 0, c.g_lens, c.g_acc,
                          c.g_pos, c.ws, c.status)
    torch.cuda.synchronize()
    assert c.status.tolist()[0] == 0 and c.status.tolist()[2] & bastion.STATUS_KV_OVERFLOW
    c.g_lens[2] = 200
    c.status.zero_()
    before[c.g_table[1:].long().flatten()] = 0
    b.bastion_paged_evict(c.g_k, c.g_v, c.g_table, c.g_lens, c.g_seen, c.g_acc, c.g_pos, 100, 0, 0, c.g_lens, c.g_acc,
                          c.g_pos, c.ws, c.status)
    torch.cuda.synchronize()
    assert c.status.tolist() == [bastion.STATUS_BAD_PAGE, 0, 0]
    after = c.g_k.clone()
    after[c.g_table[1:].long().flatten()] = 0
    assert torch.equal(before, after)


# --------------------------------------------------------------------------- together

def _decode_reference(tokens, out, q, scale):
    """Each head attends to the tokens its slots hold; tokens: {(r, h): [positions]}."""
    k_all, v_all, keep = tokens
    B, Hq, D = q.shape
    Hkv = k_all.shape[2]
    G = Hq // Hkv
    for r in range(B):
        for h in range(Hkv):
            k, v = k_all[r, keep[r][h], h].double(), v_all[r, keep[r][h], h].double()
            s = q[r, h * G:(h + 1) * G].double() @ k.T * scale
            w = s.softmax(-1)
            ds = (q[r, h * G:(h + 1) * G].double().abs() @ k.T.abs()).amax() * scale * 2.0 ** -16 + 2.0 ** -22 * s.abs().amax()
            o, size = w @ v, w @ v.abs()
            err = (out[r, h * G:(h + 1) * G].double() - o).abs()
            step = torch.finfo(out.dtype).eps / 2
            assert bool((err <= step * o.abs() * 1.01 + size * (2 * ds + 2.0 ** -14)).all()), (r, h, float(err.max()))


@pytest.mark.parametrize("graph", [False, True])
def test_budgeted_decoding(cuda_lib, graph):
    """Prompt, then steps of append, attention with weights and eviction: every step's output equals attention
    over the tokens that the slots' positions name, and the positions follow the weights."""
    from draft_tree_build_gb300 import bastion
    B, Hq, Hkv, D, budget, sink, recent = 3, 8, 2, 128, 96, 2, 16
    cache = bastion.PagedCache(B, Hq, Hkv, D, 16, 16, dev(), weights=True)
    steps, n0 = 40, torch.tensor([200, 150, 30], dtype=torch.int32)
    g = _gen(31)
    total = 200 + steps
    k_all, v_all = (torch.randn(B, total, Hkv, D, generator=g).to(BF) for _ in range(2))
    q_all = (2 * torch.randn(steps, B, Hq, D, generator=g)).to(BF)
    scale = D ** -0.5
    kd, vd, qd = k_all.to(dev()), v_all.to(dev()), q_all.to(dev())
    cache.append(kd[:, :200].contiguous(), vd[:, :200].contiguous(), n_new=n0.to(dev()))
    kt, vt = torch.zeros(B, 1, Hkv, D, dtype=BF, device=dev()), torch.zeros(B, 1, Hkv, D, dtype=BF, device=dev())
    q, out = torch.zeros(B, Hq, D, dtype=BF, device=dev()), torch.zeros(B, Hq, D, dtype=BF, device=dev())

    def step():
        cache.append(kt, vt)
        cache.attend(q, scale, out)
        cache.evict(budget, sink, recent)

    replay = step
    if graph:
        gr = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(gr):
            step()
        replay = gr.replay
    idx = torch.arange(B, device=dev())
    for t in range(steps):
        at = n0.to(dev()).long() + t
        kt.copy_(kd[idx, at][:, None])
        vt.copy_(vd[idx, at][:, None])
        q.copy_(qd[t])
        # what the step attends to: the slots' tokens, and the new one
        torch.cuda.synchronize()
        lens, pos, acc = cache.seq_len.tolist(), cache.pos.cpu(), cache.acc.cpu()
        keep = [[pos[r, h, :lens[r]].tolist() + [int(n0[r]) + t] for h in range(Hkv)] for r in range(B)]
        replay()
        torch.cuda.synchronize()
        assert cache.seq_len.tolist() == [min(budget, n + 1) for n in lens]
        assert cache.n_seen.tolist() == [int(n) + t + 1 for n in n0]
        _decode_reference((k_all, v_all, keep), out.cpu(), q_all[t], scale)
        new = cache.pos.cpu()
        for r in range(B):
            n = int(n0[r]) + t + 1
            for h in range(Hkv):
                now = new[r, h, :min(budget, lens[r] + 1)].tolist()
                assert len(set(now)) == len(now) and set(now) <= set(keep[r][h])
                must = {p for p in keep[r][h] if p < sink or p >= n - recent}
                assert must <= set(now)
                # and the slots hold those tokens' keys and values
                ids = cache.page_table[r].long()
                kk = cache.k_pool[ids].flatten(0, 1)[:len(now), h].cpu()
                vv = cache.v_pool[ids].flatten(0, 1)[:len(now), h].cpu()
                assert torch.equal(kk, k_all[r, now, h]) and torch.equal(vv, v_all[r, now, h])
    assert int(cache.status.sum()) == 0
    # the weights that stayed: a token's weight is the sum of its attention probabilities, which are positive
    live = cache.acc[:, :, :30]
    assert bool((live >= 0).all()) and bool((live.sum(-1) > 0).all())


def test_tree_step_then_commit_then_decode(cuda_lib):
    """A contiguous cache is a paged one: tree attention reads the drafted tokens' keys from it, the accepted
    path of the tree is committed, and plain decoding continues on the same memory."""
    from draft_tree_build_gb300 import bastion
    B, n_max, Hq, Hkv, D, cap = 2, 8, 8, 2, 128, 128
    cache = bastion.PagedCache(B, Hq, Hkv, D, 16, cap // 16, dev())
    g = _gen(41)
    prompt = torch.randn(B, 50, Hkv, D, generator=g).to(BF).to(dev()), torch.randn(B, 50, Hkv, D, generator=g).to(BF).to(dev())
    cache.append(*prompt, n_new=torch.tensor([50, 33], dtype=torch.int32, device=dev()))
    k_tree, v_tree = (torch.randn(B, n_max, Hkv, D, generator=g).to(BF).to(dev()) for _ in range(2))
    parent = [[-1, 0, 1, 0, 1, 2, 5, 3], [-1, 0, 0, 2, 3, 1, 5, 6]]
    anc = torch.zeros(B, n_max, 1, dtype=torch.int32)
    for r in range(B):
        for i in range(n_max):
            anc[r, i, 0] = (1 << i) | (0 if i == 0 else int(anc[r, parent[r][i], 0]))
    kc, vc = cache.contiguous()
    assert kc.data_ptr() == cache.k_pool.data_ptr()
    ctx = cache.seq_len.clone()
    for r in range(B):
        n = int(ctx[r])
        kc[r, n:n + n_max], vc[r, n:n + n_max] = k_tree[r], v_tree[r]
    q = torch.randn(B, n_max, Hq, D, generator=g).to(BF).to(dev())
    out = torch.zeros_like(q)
    ws = bastion.workspace(bastion.bastion_tree_attention_workspace_bytes(B, n_max, Hq, Hkv, D, cap), dev())
    nn = torch.full((B,), n_max, dtype=torch.int32, device=dev())
    bastion.bastion_tree_attention(q, kc, vc, ctx, nn, anc.to(dev()), D ** -0.5, out, ws, cache.status)
    path = torch.tensor([[0, 1, 2, 5, -1], [0, 2, -1, -1, -1]], dtype=torch.int32, device=dev())  # accept_nodes
    tip = [5, 2]
    cache.append(k_tree, v_tree, rows=path)
    torch.cuda.synchronize()
    assert cache.seq_len.tolist() == [54, 35] and int(cache.status.sum()) == 0
    # decoding the tip's query over the committed path sees what the tree's row saw
    q1 = torch.stack([q[r, tip[r]] for r in range(B)]).contiguous()
    o1, lse = torch.empty_like(q1), torch.empty(B, Hq, device=dev())
    cache.attend(q1, D ** -0.5, o1, lse)
    torch.cuda.synchronize()
    ref.check_attention(o1, lse, q1, cache.k_pool, cache.v_pool, cache.page_table, cache.seq_len.cpu(), D ** -0.5)
    o_tree = torch.stack([out[r, tip[r]] for r in range(B)])
    assert float((o1.float() - o_tree.float()).abs().max()) < 2e-2
