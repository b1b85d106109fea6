"""The operators of a layer's step together, as a serving loop uses them: pages and slots for the step's tokens, norm
and rotation with keys and values stored, attention over a shared prefix and the own slots; captured in a graph."""
import math

import pytest
import torch

import layerref as ref
import pagedref
from gpuhelp import dev

pytestmark = pytest.mark.gpu


class Loop:
    """A cache whose requests share two prompts, and plain copies of everything on the CPU."""
    B, Hq, Hkv, D, page, m = 7, 8, 2, 128, 16, 4

    def __init__(self, dtype, seed=0):
        from draft_tree_build_gb300 import bastion
        self.b, self.g = bastion, torch.Generator().manual_seed(seed)
        B, D = self.B, self.D
        self.dtype, self.plens, self.start = dtype, [200, 77], [0, 4, 6]  # the last request has no prefix
        pre = [-(-n // self.page) for n in self.plens]
        self.cache = bastion.PagedCache(B, self.Hq, self.Hkv, D, self.page, 8, dev(), dtype, n_pages=60, new_tokens=200,
                                        reserved=sum(pre), prefixes=2)
        self.prefix_table = torch.zeros(2, max(pre), dtype=torch.int32)
        self.prefix_table[0, :pre[0]], self.prefix_table[1, :pre[1]] = torch.arange(pre[0]), torch.arange(pre[0], sum(pre))
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev())  # noqa: E731
        self.pt, self.pl, self.gs = self.prefix_table.to(dev()), i32(self.plens), i32(self.start)
        self.freq, self.factor = bastion.rope_frequencies(D, 1e6, dev(), "yarn", 4.0, low=1.0, high=32.0)
        self.qw, self.kw = (torch.randn(D, generator=self.g).to(dtype).to(dev()) for _ in range(2))
        self.scale = ref.scale_of(D)
        self.keys = [[] for _ in range(B)]  # what each request's slots hold

    def rows(self, T):
        x = torch.randn(T, self.Hq + 2 * self.Hkv, self.D, generator=self.g).to(self.dtype).to(dev())
        return x[:, :self.Hq], x[:, self.Hq:self.Hq + self.Hkv], x[:, self.Hq + self.Hkv:]

    def fill_prefixes(self):
        """The prompts go through the same kernel, with slots of the reserved pages."""
        T = sum(self.plens)
        slots = torch.cat([self.prefix_table[g][torch.arange(n) // self.page] * self.page + torch.arange(n) % self.page
                           for g, n in enumerate(self.plens)]).long().to(dev())
        pos = torch.cat([torch.arange(n) for n in self.plens]).to(torch.int32).to(dev())
        q, k, v = self.rows(T)
        out = torch.empty(T, self.Hq, self.D, dtype=self.dtype, device=dev())
        self.cache.write(q, k, v, pos, slots, self.freq, out, self.qw, self.kw, factor=self.factor)

    def step(self, m, n_new, q, k, v, q_out, trim=False):
        slots, pos = self.cache.reserve(m, n_new, trim=trim)
        self.cache.write(q, k, v, pos, slots, self.freq, q_out, self.qw, self.kw, factor=self.factor)

    def attend(self, q, out, lse):
        self.cache.attend_shared(q, self.pt, self.pl, self.gs, self.scale, out, lse)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("graph", [False, True])
def test_decoding_behind_shared_prompts(cuda_lib, dtype, graph):
    L = Loop(dtype)
    c, B = L.cache, L.B
    L.fill_prefixes()
    # the requests' own prompts, of mixed lengths; one request has none yet
    count = torch.tensor([30, 1, 16, 0, 45, 17, 60], dtype=torch.int32)
    q, k, v = L.rows(B * 60)
    out0 = torch.full((B * 60, L.Hq, L.D), 7.0, dtype=dtype, device=dev())
    L.step(60, count.to(dev()), q, k, v, out0)
    torch.cuda.synchronize()
    assert c.seq_len.tolist() == count.tolist() and c.held.tolist() == [-(-n // 16) for n in count.tolist()]
    want, size = ref.norm_rope(q, L.qw, 1e-6, c.slot_pos[:B * 60].clamp(min=0), L.freq, L.D, False, L.factor)
    live = c.slot_pos[:B * 60] >= 0
    assert int(live.sum()) == int(count.sum()) and bool((out0[~live] == 7).all())
    ref.check_norm_rope(out0[live], want[live], size[live])

    one = torch.ones(B, dtype=torch.int32, device=dev())
    q1, k1, v1 = L.rows(B)
    q1, k1, v1 = q1.clone(), k1.clone(), v1.clone()
    turned = torch.zeros(B, L.Hq, L.D, dtype=dtype, device=dev())
    out, lse = torch.zeros_like(turned), torch.zeros(B, L.Hq, device=dev())

    def step():
        L.step(1, one, q1, k1, v1, turned, trim=True)
        L.attend(turned, out, lse)

    if graph:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
    lens = count.tolist()
    for i in range(30):
        for x, y in zip((q1, k1, v1), L.rows(B)):
            x.copy_(y)
        if i == 20:  # request 1 ends: its pages go back, and it starts anew
            c.seq_len[1] = 0
            lens[1] = 0
        g.replay() if graph else step()
        torch.cuda.synchronize()
        lens = [n + 1 for n in lens]
        assert c.seq_len.tolist() == lens and not bool(c.status.any()) and int(c.write_status) == 0
        held = [-(-n // 16) for n in lens]
        assert c.held.tolist() == held and int(c.n_free) == 60 - 18 - sum(held)
        table = c.page_table.cpu()
        used = [p for r in range(B) for p in table[r, :held[r]].tolist()]
        assert len(set(used)) == len(used) and min(used) >= 18  # a page belongs to one request, and none to a prefix
        # the step's rows, turned by their own positions
        pos = torch.tensor(lens, dtype=torch.int32, device=dev()) - 1
        for x, w, got in ((q1, L.qw, turned), (k1, L.kw, None)):
            want, size = ref.norm_rope(x, w, 1e-6, pos, L.freq, L.D, False, L.factor)
            if got is None:
                at = [int(table[r, (lens[r] - 1) // 16]) for r in range(B)]
                got = c.k_pool[at, [(n - 1) % 16 for n in lens]]
                assert torch.equal(c.v_pool[at, [(n - 1) % 16 for n in lens]], v1)
            ref.check_norm_rope(got, want, size)
        if i % 7 == 0 or i == 20:
            k, v, t, n = ref.joined(c.k_pool, c.v_pool, table, lens, L.prefix_table, L.plens, L.start)
            pagedref.check_attention(out, lse, turned, k, v, t, n, L.scale)


def test_running_out_of_pages_and_packed_prompts(cuda_lib):
    """Requests that find no page keep their lengths, and get them once others have ended."""
    from draft_tree_build_gb300 import bastion
    c = bastion.PagedCache(4, 4, 2, 64, 8, 10, dev(), n_pages=20, new_tokens=64)
    slots, pos = c.reserve(64, torch.tensor([60, 40, 50, 0], dtype=torch.int32, device=dev()), packed=True, n_rows=160)
    torch.cuda.synchronize()
    # 8 + 5 + 7 pages: all twenty
    assert c.status.tolist() == [0, 0, 0, 0] and int(c.n_free) == 0 and c.row_start.tolist() == [0, 60, 100, 150, 150]
    assert slots.tolist()[150:] == [-1] * 10 and sorted(set(s // 8 for s in slots.tolist()[:150])) == list(range(20))
    assert pos.tolist()[60:100] == list(range(40))
    c.reserve(5, torch.tensor([1, 1, 5, 3], dtype=torch.int32, device=dev()))
    torch.cuda.synchronize()
    assert c.status.tolist() == [0, 256, 0, 256] and c.seq_len.tolist() == [61, 40, 55, 0]
    c.status.zero_()
    c.seq_len[0] = 0
    c.reserve(5, torch.tensor([0, 1, 5, 3], dtype=torch.int32, device=dev()), trim=True)
    torch.cuda.synchronize()
    assert c.status.tolist() == [0] * 4 and c.seq_len.tolist() == [0, 41, 60, 3] and int(c.n_free) == 20 - 6 - 8 - 1
    assert c.held.tolist() == [0, 6, 8, 1]


def test_a_drafted_tree_is_turned_by_its_positions(cuda_lib):
    """Keys of a tree's nodes, turned by depth, in a contiguous cache behind its context: tree attention over them, and
    the accepted path's rows into the paged cache, are those of the plain turn."""
    from draft_tree_build_gb300 import bastion
    g = torch.Generator().manual_seed(3)
    B, n_max, Hq, Hkv, D, L_cap, page = 3, 16, 8, 2, 128, 96, 16
    ctx, nodes = torch.tensor([40, 7, 0], dtype=torch.int32), torch.tensor([16, 5, 9], dtype=torch.int32)
    parent = torch.full((B, n_max), -1, dtype=torch.int32)
    depth, mask = torch.zeros(B, n_max, dtype=torch.int32), torch.zeros(B, n_max, 1, dtype=torch.int32)
    for r in range(B):
        mask[r, 0] = 1
        for i in range(1, n_max):
            p = int(torch.randint(0, i, (1,), generator=g))
            parent[r, i], depth[r, i], mask[r, i] = p, depth[r, p] + 1, mask[r, p] | (1 << i)
    pos = (ctx[:, None] + depth).masked_fill(torch.arange(n_max) >= nodes[:, None], -7)
    x = torch.randn(B, n_max, Hq + 2 * Hkv, D, generator=g).bfloat16().to(dev())
    k_cache, v_cache = (torch.randn(B, L_cap, Hkv, D, generator=g).bfloat16().to(dev()) for _ in range(2))
    rows = x.view(B * n_max, Hq + 2 * Hkv, D)
    # slot ctx + i of request r of a contiguous cache
    i = torch.arange(n_max)
    slots = (torch.arange(B)[:, None] * L_cap + ctx[:, None] + i).masked_fill(i >= nodes[:, None], -1)
    freq, _ = bastion.rope_frequencies(D, 1e6, dev())
    q = torch.zeros(B, n_max, Hq, D, dtype=torch.bfloat16, device=dev())
    k_rows = torch.zeros(B, n_max, Hkv, D, dtype=torch.bfloat16, device=dev())
    st = torch.zeros(1, dtype=torch.int32, device=dev())
    pools = [t.view(B * L_cap // page, page, Hkv, D) for t in (k_cache, v_cache)]
    bastion.bastion_qk_norm_rope(rows[:, :Hq], rows[:, Hq:Hq + Hkv], pos.view(-1).to(dev()), freq, q.view(-1, Hq, D), st,
                                 k_out=k_rows.view(-1, Hkv, D), v=rows[:, Hq + Hkv:], k_pool=pools[0], v_pool=pools[1],
                                 slots=slots.view(-1).to(dev()))
    out, status = torch.zeros_like(q), torch.zeros(B, dtype=torch.int32, device=dev())
    ws = bastion.workspace(bastion.bastion_tree_attention_workspace_bytes(B, n_max, Hq, Hkv, D, L_cap), dev())
    bastion.bastion_tree_attention(q, k_cache, v_cache, ctx.to(dev()), nodes.to(dev()), mask.to(dev()), ref.scale_of(D), out,
                                   ws, status)
    torch.cuda.synchronize()
    assert int(st) == 0 and not bool(status.any())
    want_k, size = ref.norm_rope(x[:, :, Hq:Hq + Hkv].reshape(-1, Hkv, D), None, 0, pos.view(-1).to(dev()), freq, D, False, 1.0)
    live = (pos >= 0).view(-1).to(dev())
    ref.check_norm_rope(k_rows.view(-1, Hkv, D)[live], want_k[live], size[live])
    for r in range(B):
        n, c = int(nodes[r]), int(ctx[r])
        assert torch.equal(k_cache[r, c:c + n], k_rows[r, :n])
        for j in range(n):
            see = list(range(c)) + [c + t for t in range(n) if int(mask[r, j, 0]) >> t & 1]
            k, v = k_cache[r, see].double().repeat_interleave(4, 1), v_cache[r, see].double().repeat_interleave(4, 1)
            w = torch.softmax(torch.einsum("hd,lhd->hl", q[r, j].double(), k) * ref.scale_of(D), -1)
            o = torch.einsum("hl,lhd->hd", w, v)
            assert float((out[r, j].double() - o).abs().max()) < 2e-2


def test_the_cache_refuses(cuda_lib):
    from draft_tree_build_gb300 import bastion
    make = lambda **kw: bastion.PagedCache(2, 4, 2, 64, 8, 4, dev(), **kw)  # noqa: E731
    with pytest.raises(bastion.BastionError, match="new_tokens"):
        make().reserve(1)
    with pytest.raises(bastion.BastionError, match="new_tokens"):
        make(new_tokens=2).reserve(3)
    with pytest.raises(bastion.BastionError, match="prefixes"):
        make().attend_shared(*[None] * 6)
    with pytest.raises(bastion.BastionError, match="weights"):
        make(new_tokens=2, weights=True)
    with pytest.raises(bastion.BastionError, match="reserved"):
        make(new_tokens=2, n_pages=4, reserved=4)
    with pytest.raises(bastion.BastionError, match="order"):
        make(new_tokens=2).contiguous()
    # another stream than the current one
    s = torch.cuda.Stream()
    c = make(new_tokens=2)
    torch.cuda.synchronize()
    slots, pos = c.reserve(2, stream=s)
    s.synchronize()
    assert pos.tolist() == [0, 1, 0, 1] and math.prod(slots.shape) == 4


def test_one_workspace_serves_all_calls(cuda_lib):
    """Plan, append, one-token attention, eviction and shared-prefix attention in turn on one workspace, in two orders."""
    from draft_tree_build_gb300 import bastion
    from test_gpu_paged import Case
    from test_gpu_plan import EDGES, Plan
    from test_gpu_prefix import Prefix
    long_own, short_own = Prefix([9000, 40], [9, 30], [100] * 39, 8, 2, seed=1), Prefix([700], [5], [9] * 5, 8, 2, 64, seed=2)
    plan, att = Plan(EDGES, 17), Case([5000, 20, 300], 8, 2, weights=True, seed=3)
    ws = max((x.ws for x in (long_own, short_own, plan, att)), key=lambda t: t.numel())
    ws = bastion.workspace(ws.numel(), dev())
    plan.ws = ws
    for turn in range(6):
        calls = [lambda: long_own.run(ws), plan.run, lambda: att.run(ws), lambda: short_own.run(ws)]
        for f in calls if turn % 2 else calls[::-1]:
            f()
        torch.cuda.synchronize()
        for x in (long_own, short_own, att):
            x.check()
            x.out.fill_(7.0)
        want = ref.plan(plan.table, stack=plan.stack, **plan.args)
        assert plan.slots.tolist() == want["slots"] and plan.t["table"].tolist() == want["table"]
        plan.slots.fill_(77)


def test_many_calls_of_large_batches_agree(cuda_lib):
    """Tiles overwritten while they are read would show as differences between calls: 1,024 rows a KV head, all SMs busy."""
    from test_gpu_prefix import Prefix
    p = Prefix([20000], [128], [32] * 128, 16, 2, 128, 64, "slot", seed=7)
    p.run().check()
    out, lse = p.out.clone(), p.lse.clone()
    for i in range(50):
        p.out.zero_()
        p.run()
        assert torch.equal(p.out, out) and torch.equal(p.lse, lse), i
